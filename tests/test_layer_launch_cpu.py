"""The launches of the short convolution, the selective scan with heads and the norm with
rotation against a stand-in for the CUDA runtime (see test_launch_cpu)."""

from test_launch_cpu import child  # noqa: F401

BODY = """
lib.lr_selective_heads_workspace_size.restype = ctypes.c_size_t


def heads(io, B, L, H, P, N):
    n = lib.lr_selective_heads_workspace_size(I(B), I(L), I(H), I(1), I(P), I(N), io)
    return lib.lr_selective_heads_fwd(p(), I(H * P), p(), I(H), p(), I(N), p(), I(N), p(), I(H * P), p(), p(), p(), None,
                                      p(), p(), p(), I(B), I(L), I(H), I(1), I(P), I(N), io, 1, p(), ctypes.c_size_t(n),
                                      None)


def heads_step(io, N):
    return lib.lr_selective_heads_step(p(), I(128), p(), I(2), p(), I(N), p(), I(N), None, I(0), p(), None, None, p(), p(),
                                       p(), I(3), I(2), I(1), I(64), I(N), io, 1, None)


def conv(io, L, C, W):
    return lib.lr_causal_conv_fwd(p(), I(C), p(), p(), p(), None, p(), p(), I(2), I(L), I(C), I(W), 1, io, None)


def conv_step(io, C):
    return lib.lr_causal_conv_step(p(), I(C), p(), p(), p(), p(), p(), I(2), I(C), I(4), 0, io, None)


def rope(io, d, rot, pairs):
    return lib.lr_head_norm_rope(p(), I(4 * d), p(), I(2 * d), p(), p(), p(), p(), p(), p(), I(9), I(4), I(2), I(d), I(rot),
                                 1, F(1e-6), pairs, io, None)


# (call, its launches): gates and scan; with segments; with the states' columns in parts; the
# CUDA cores in one launch and in segments
calls = [(lambda: heads(BF16, 1, 77, 4, 128, 128), 2), (lambda: heads(BF16, 1, 16384, 2, 64, 64), 3),
         (lambda: heads(BF16, 1, 77, 4, 64, 192), 3), (lambda: heads(F32, 1, 40, 4, 128, 128), 1),
         (lambda: heads(F32, 1, 9000, 1, 64, 64), 2), (lambda: heads(BF16, 1, 9, 4, 64, 64), 1),
         (lambda: heads_step(BF16, 128), 1), (lambda: heads_step(F32, 33), 1), (lambda: conv(BF16, 999, 512, 4), 1),
         (lambda: conv(F32, 5, 33, 2), 1), (lambda: conv_step(BF16, 512), 1), (lambda: conv_step(F32, 33), 1),
         (lambda: rope(BF16, 128, 128, 0), 1), (lambda: rope(F32, 80, 64, 1), 1), (lambda: rope(F32, 33, 32, 0), 1),
         (lambda: rope(F32, 512, 512, 0), 1), (lambda: rope(BF16, 511, 510, 1), 1)]
"""


def test_launches(child):  # noqa: F811
    child(BODY + """
for i, (call, n) in enumerate(calls):
    assert run(call) == (0, n), (i, run(call))
    fake.fake_set_pending_error(201)   # an older unread error is not the call's
    assert run(call) == (0, n), i
    for k in range(1, n + 1):
        fake.fake_fail_next_launch(k)
        assert run(call) == (-5, k - 1), (i, k)
""")


def test_every_device_of_a_process(child):  # noqa: F811
    child(BODY + """
for dev in (0, 3, 0, 1):
    fake.fake_set_device(dev)
    for i, (call, n) in enumerate(calls):
        assert run(call) == (0, n), (dev, i)
fake.fake_set_device(4)
fake.fake_fail_next_attribute()
assert calls[0][0]() == -5 and calls[0][0]() == 0
""")
