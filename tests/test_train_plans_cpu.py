"""The shapes of test_train_tiles_gpu.py meet every instantiation of the training kernels: a
change of the planners that leaves one without a test fails here."""

import train_plans


def test_every_kernel_is_met():
    import w4a16_int4_weight_amd as w
    missing = train_plans.every_kernel() - train_plans.met(w)
    assert not missing, sorted(missing, key=str)


def test_the_sizes_leave_a_rest():
    for M, K, N in train_plans.GEMM_GRAD + train_plans.GATED + train_plans.LOSS:
        assert N % 16 == 8 and K % 128 == 0
    for shapes in (train_plans.GEMM_GRAD, train_plans.GATED, train_plans.LOSS):
        assert {M % 16 for M, _, _ in shapes} - {0}, shapes
