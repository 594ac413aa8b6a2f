"""The launches of the C entry points against a stand-in for the CUDA runtime
(fake_cudart.c, preloaded in a child process; nothing runs on a GPU and the
pointers are never dereferenced): what a call answers where a launch fails, where an
older error of the thread was never read, and on the second device of a process."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

PRELUDE = """
import ctypes, os, sys
fake = ctypes.CDLL(os.environ["LD_PRELOAD"])
lib = ctypes.CDLL(sys.argv[1])
P, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
p = lambda: P(0x7F0000000000)
lib.lr_decay_attn_workspace_size.restype = ctypes.c_size_t
lib.lr_hgrn2_workspace_size.restype = ctypes.c_size_t
F32, BF16 = 0, 1


def prompt(io, B, L, H, dk, dv):
    n = lib.lr_decay_attn_workspace_size(I(B), I(L), I(H), I(H), I(dk), I(dv), io)
    return lib.lr_decay_attn_fwd(p(), p(), p(), p(), p(), None, F(1), p(), p(), p(), I(B), I(L), I(H), I(H), I(dk),
                                 I(dv), io, p(), ctypes.c_size_t(n), None)


def step(io, dk):
    return lib.lr_decay_attn_step(p(), p(), p(), p(), p(), F(1), p(), p(), p(), I(2), I(4), I(4), I(dk), I(64), io, None)


def norm(io, C, G):
    return lib.lr_group_norm_act(p(), p(), p(), p(), p(), I(8), I(C), I(G), F(1e-5), 0, io, None)


def hgrn2(io):
    n = lib.lr_hgrn2_workspace_size(I(1), I(64), I(2), I(128), I(128), io)
    return lib.lr_hgrn2_fwd(p(), p(), p(), p(), p(), p(), p(), I(1), I(64), I(2), I(128), I(128), I(64), io, p(),
                            ctypes.c_size_t(n), None)


# (call, its launches): one launch, segments, key columns in parts, both kernels
decay = [(lambda: prompt(BF16, 1, 77, 4, 128, 128), 1), (lambda: prompt(BF16, 1, 16384, 2, 64, 64), 2),
         (lambda: prompt(BF16, 1, 77, 4, 192, 64), 2), (lambda: prompt(F32, 1, 40, 4, 128, 128), 1),
         (lambda: prompt(F32, 1, 9000, 1, 64, 64), 2), (lambda: prompt(F32, 2, 40, 64, 300, 64), 1),
         (lambda: step(BF16, 128), 1), (lambda: step(F32, 33), 1), (lambda: norm(BF16, 512, 4), 1),
         (lambda: norm(F32, 99, 3), 1), (lambda: norm(F32, 4096, 1), 1)]


def run(call):
    before = fake.fake_launches()
    rc = call()
    return rc, fake.fake_launches() - before
"""


@pytest.fixture(scope="module")
def child(tmp_path_factory):
    from selective_state_space_chunked_gb300 import build
    lib = build.build()
    so = str(tmp_path_factory.mktemp("fake") / "fake_cudart.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", os.path.join(HERE, "fake_cudart.c"), "-o", so], check=True)

    def run(body):
        r = subprocess.run([sys.executable, "-c", PRELUDE + body, lib], env={**os.environ, "LD_PRELOAD": so}, cwd=ROOT,
                           capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
    return run


def test_every_call_launches_what_it_should(child):
    child("""
for i, (call, n) in enumerate(decay):
    assert run(call) == (0, n), (i, run(call))
""")


def test_an_older_unread_error_is_not_the_calls(child):
    """A call whose launches succeeded answers LR_OK: a caller that is told of a
    failure would launch again, onto a state that has already been updated."""
    child("""
for i, (call, n) in enumerate(decay):
    fake.fake_set_pending_error(201)
    assert run(call) == (0, n), i
""")


def test_a_failed_launch_is_reported(child):
    child("""
for i, (call, n) in enumerate(decay):
    for k in range(1, n + 1):
        fake.fake_fail_next_launch(k)
        assert run(call) == (-5, k - 1), (i, k)
    assert run(call) == (0, n), i
""")


def test_every_device_of_a_process(child):
    """Limits on a kernel's shared memory are a device's own, and a device where
    setting one failed is tried again."""
    child("""
for dev in (0, 3, 0, 1):
    fake.fake_set_device(dev)
    for i, (call, n) in enumerate(decay):
        assert run(call) == (0, n), (dev, i)
    for io in (BF16, F32):
        assert hgrn2(io) == 0, (dev, io)
for dev, call in ((4, decay[0][0]), (5, lambda: hgrn2(BF16)), (6, lambda: hgrn2(F32))):
    fake.fake_set_device(dev)
    fake.fake_fail_next_attribute()
    assert call() == -5 and call() == 0, dev
""")
