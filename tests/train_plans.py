"""The host planners of the training operators, as the library exports them, and which
instantiation of a kernel a call takes."""

import ctypes


class _Product(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("mr", "sub", "tiles_m", "tiles_n", "splits")] + [("bytes", ctypes.c_size_t)]


class _Grad(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("bm", "tiles_m", "tiles_k", "splits")] + [("bytes", ctypes.c_size_t)]


_i64, _bool = ctypes.c_int64, ctypes.c_bool


def _function(w, symbol, restype, argtypes):
    f = w.lib[symbol]
    f.restype, f.argtypes = restype, argtypes
    return f


def product(w, M, K, cols, G, gated):
    """`cols` columns of the weight (2F of a gated block)"""
    f = _function(w, "_ZN5w4a1612plan_productEllllb", _Product, [_i64] * 4 + [_bool])
    return f(M, K, cols, K if G == -1 else G, gated)


def grad(w, M, K, n, forced=False):
    return _function(w, "_ZN5w4a169plan_gradElllb", _Grad, [_i64] * 3 + [_bool])(M, K, n, forced)


def small(w, M, K):
    return _function(w, "_ZN5w4a1613small_productEll", _bool, [_i64] * 2)(M, K)


def sub(G):
    return 128 // G if 0 < G < 128 else 1


def loss_piece(w, M, V):
    """columns of the vocabulary that a loss with a gradient takes at a time (M up to 4096)"""
    most = max((1 << 28) // (2 * M) // 512 * 512, 512)
    pieces = -(-V // most)
    piece = (-(-V // pieces) + 511) // 512 * 512
    return piece if V > piece else V


def kernels(w, op, M, K, N, dtype, G):
    """The instantiations a call meets: ("small", op, dtype, sub, row blocks a wave),
    ("tile", op, dtype, sub, row fragments, whether K is split) and ("grad", op, dtype, sub, tile rows, whether
    the sum is split). N: F of a gated block, V of a head."""
    def tile(p):
        return p.mr, p.splits > 1
    s, out = sub(G), set()
    gated = op in ("gated", "gated_grad")
    cols = 2 * N if gated else N
    if op != "gemm_grad":
        few = small(w, M, K) and op != "ce_grad"
        if few:
            jp = -(-(K // 128) // 8)
            out.add(("small", op, dtype, s, jp if jp <= 2 else 4))
        elif op == "ce_grad":
            out.add(("tile", op, dtype, s, *tile(product(w, M, K, loss_piece(w, M, N), G, False))))
        else:
            out.add(("tile", op, dtype, s, *tile(product(w, M, K, cols, G, gated))))
    if op in ("gemm_grad", "gated_grad"):
        p = grad(w, M, K, cols)
        out.add(("grad", op, dtype, s, p.bm, p.splits > 1))
    elif op == "ce_grad":
        p = grad(w, M, K, loss_piece(w, M, N), True)
        out.add(("grad", op, dtype, s, p.bm, True))
    return out


# Shapes (M, K, columns of a half or of the head) that between them meet every instantiation,
# with sizes that leave a rest in the last tile of rows, of columns and of W^T's columns.
GEMM_GRAD = [(1, 384, 392), (5, 384, 520), (2100, 384, 392), (1030, 384, 520), (3001, 640, 392), (2100, 384, 648),
             (1800, 2176, 392), (2100, 384, 2728), (1800, 4480, 392), (515, 4480, 2728)]
GATED = [(1, 384, 200), (7, 384, 264), (13, 1152, 264), (16, 2176, 136), (11, 4224, 200), (3, 4224, 16392), (17, 384, 200),
         (17, 1152, 200), (2100, 384, 200), (1030, 384, 264), (2100, 896, 200), (1030, 384, 648), (1800, 2176, 200),
         (3001, 384, 264), (1500, 2176, 264), (3001, 384, 648), (3001, 384, 1000), (3001, 4224, 264), (1800, 4480, 200),
         (129, 384, 33000)]
LOSS = [(1, 384, 24), (16, 1152, 200), (7, 2176, 264), (9, 4224, 264), (3, 4224, 33000), (17, 384, 136), (17, 1152, 264),
        (2100, 384, 40), (3001, 640, 136), (3001, 384, 520), (4095, 2176, 40), (1800, 2176, 72), (1800, 384, 2056),
        (1800, 4480, 40), (4095, 5248, 264)]
GROUPS = [128, 64, 32]
DTYPES = ["bf16", "fp16"]


def every_kernel():
    """What the shapes above have to meet."""
    out = set()
    for d in DTYPES:
        for G in GROUPS:
            s = sub(G)
            out |= {("small", op, d, s, jp) for op in ("gated", "gated_grad", "ce") for jp in (1, 2, 4)}
            out |= {("tile", op, d, s, mr, split) for op in ("gated", "gated_grad", "ce", "ce_grad")
                    for mr in ((1, 2, 4, 8) if s == 1 else (1, 2, 4)) for split in (False, True)}
            out |= {("grad", op, d, s, bm, split) for op in ("gemm_grad", "gated_grad") for bm in (16, 32, 64, 128, 256)
                    for split in (False, True)}
            out |= {("grad", "ce_grad", d, s, bm, True) for bm in (16, 32, 64, 128, 256)}
    return out


def met(w):
    out = set()
    for d in DTYPES:
        for G in GROUPS:
            for op, shapes in (("gemm_grad", GEMM_GRAD), ("gated", GATED), ("gated_grad", GATED), ("ce", LOSS), ("ce_grad", LOSS)):
                for M, K, N in shapes:
                    out |= kernels(w, op, M, K, N, d, G)
    return out
