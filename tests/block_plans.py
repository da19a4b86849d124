"""Shapes (M, K, N) and (M, K, F) that between them take every kernel form of every product of the
layer operators: forward, dx and the weight gradients, by the few-token kernel with each count
of tokens and slices and by CTA pairs with each tile. tests/test_block_plans.py holds them to it."""
import ctypes

from linear_cross_entropy_gemm_gb300 import _lib

LINEAR = [(1, 72, 41), (1, 224, 67), (147, 80, 41), (1, 7960, 771), (131, 9816, 45), (8443, 96, 129),
          (3325, 4664, 47), (17, 104, 43), (35, 72, 43), (19, 248, 69), (35, 224, 71), (17, 584, 203),
          (35, 520, 211), (67, 72, 10467), (1931, 80, 1769), (10655, 136, 243), (275, 1928, 1625),
          (65, 6344, 4839), (261, 4224, 3219), (1, 8, 481), (17, 8, 491), (55, 8, 463),
          (6247, 1608, 41), (91, 13608, 16136)]
GATED = [(1, 72, 40), (1, 208, 72), (1, 1256, 296), (1389, 72, 40), (29, 15488, 40), (145, 5664, 40),
         (3169, 2512, 40), (17, 72, 72), (37, 96, 40), (35, 200, 88), (17, 200, 216), (33, 544, 232),
         (71, 80, 2904), (1943, 72, 632), (9855, 168, 104), (2361, 152, 888), (73, 5296, 2536),
         (131, 6104, 1688), (75, 15800, 11112), (69, 112, 40), (1, 80, 10440), (27, 72, 10040),
         (41, 72, 9800), (7581, 1608, 40), (69, 4304, 9448)]
PRODUCTS = ("forward", "dx", "dW")


def plans(op, M, K, N):
    """(product, few_tokens, halves, columns, slices) of the three products."""
    lib = _lib.load()
    if op == "linear":
        p, ask = _lib.FlceLinearParams(M=M, K=K, N=N), lib.flce_linear_plan
    else:
        p, ask = _lib.FlceGatedParams(M=M, K=K, F=N), lib.flce_gated_plan
    out = []
    for i, product in enumerate(PRODUCTS):
        plan = _lib.FlcePlan()
        assert ask(ctypes.byref(p), i, ctypes.byref(plan)) == 0
        out.append((product, plan.few_tokens, plan.halves, plan.columns, plan.slices))
    return out
