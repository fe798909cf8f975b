"""dense_fp32_gemm_amd -- dense FP32 GEMM for AMD MI355X (gfx950, CDNA4).

C[M x N] = A[M x K] . B[K x N], row-major, any M/N/K, computed by hand-written
HIP kernels on the FP32 matrix cores behind the C-ABI library
``libgemm_f32.so`` (declared in ``include/gemm_f32.h``).  ``binding`` is the
ctypes layer with the same names; ``inputs`` holds the seeded operand
generators.  The binding loads the library on first use.

``include/gemm_f32_rows.h`` adds products whose second matrix is chosen row by
row (binary32, bfloat16, half): routing to experts, the experts' products, their
gradients and weighted sums, and low-rank adapters; ``binding`` has them as
functions of torch tensors (``route``, ``expert_map``, ``grouped_matmul``,
``combine``, ``adapter_matmul`` and the ``*_grad`` ones).

``include/gemm_f32_ffn.h`` adds the operators around a feed-forward block's products:
the root-mean-square norm with the residual's addition and its gradient, rows in 8
bits and their product with 8-bit weights, and the gated pair of projections, dense
or by expert, with its gradient (``rms_norm``, ``rms_norm_int8``, ``rms_norm_grad``,
``quantize``, ``int8_matmul``, ``gated_matmul``, ``gate_grad``).
"""
