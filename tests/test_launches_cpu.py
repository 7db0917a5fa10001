"""What the host side of the 8-bit cache's operators launches, and on what conditions, without a GPU: the library's objects are linked
with a stand-in for the CUDA runtime (launch_record.c) that records launches."""
import ctypes
import glob
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

from transformer_head_scaled_fwd_gb300 import binding as bnd  # noqa: E402
from transformer_head_scaled_fwd_gb300 import build as B  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))
P = ctypes.c_void_p(4096)


class Record(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("cluster", ctypes.c_uint),
                ("smem", ctypes.c_int), ("allowed", ctypes.c_int), ("portable", ctypes.c_int)]


@pytest.fixture(scope="module")
def linked(tmp_path_factory):
    if shutil.which("g++") is None or shutil.which("gcc") is None:
        pytest.skip("no host compiler")
    B.build()
    objects = sorted(glob.glob(os.path.join(B.BUILD, "*.cu.o")))
    if [os.path.basename(o)[:-2] for o in objects] != [os.path.basename(s) for s in B._sources()]:
        B.build(force=True)
        objects = sorted(glob.glob(os.path.join(B.BUILD, "*.cu.o")))
    at = tmp_path_factory.mktemp("launches")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B._nvcc()))), "include")
    subprocess.run(["gcc", "-O1", "-fPIC", "-I", cuda, "-c", os.path.join(HERE, "launch_record.c"), "-o", str(at / "record.o")], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", str(at / "lib.so"), *objects, str(at / "record.o"), "-Wl,-z,defs"], check=True)
    return at


class Recorded:
    """A library of its own, so that what it keeps a device is asked again."""

    def __init__(self, at, name, sms=152, cluster=16):
        path = str(at / f"{name}.so")
        shutil.copy(str(at / "lib.so"), path)
        self.lib = ctypes.CDLL(path)
        os.remove(path)
        self.lib.fake_device(sms, cluster)
        vp, i, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        self.lib.mha_last_error.restype = ctypes.c_char_p
        self.lib.mha_coded_append.argtypes = [i] + [vp] * 10 + [i] * 5 + [vp] * 5
        self.lib.mha_paged_resize.argtypes = [vp, vp, i, i, vp, i64, i, vp, i, vp, vp, vp, i, vp, vp]

    def _launched(self, status):
        assert status == 0, self.lib.mha_last_error()
        at = ctypes.POINTER(Record)()
        n = self.lib.fake_records(ctypes.byref(at))
        got = [Record.from_buffer_copy(at[j]) for j in range(n)]
        self.lib.fake_clear()
        return got

    def append(self, dt=1, n=4, T=64, h=8, h_kv=2, d=128, rot=64, interleaved=0, block=16, code=0):
        page = max(block, 64 // block * block)
        strides = ctypes.byref(bnd.StridesT(T * 4096, 4096, 128))
        pages = bnd.PagedCacheT(4096, 4096, page * 4096, 4096, 128, 1000, page, 4096, 64, 64)
        cache = ctypes.byref(bnd.CodedCacheT(pages, code, block, 4096, 4096))
        rotary = ctypes.byref(bnd.RotaryT(inv_freq=4096, rot_dim=rot, interleaved=interleaved, scale=1.0)) if rot else None
        got = self._launched(self.lib.mha_coded_append(dt, P, strides, P, strides, P, strides, None, None, P, strides, n, T, h, h_kv, d, P,
                                                       None, rotary, cache, None))
        assert len(got) == 1
        return got[0]


def test_an_appends_shared_memory_limit_is_never_lowered(linked):
    """The limit is state of the kernel in the whole process: a call that sets less than another one needs makes that one's launch fail,
    if its own setting came before and its launch comes after."""
    r = Recorded(linked, "limit")
    limits, most = {}, {}
    for dt in (0, 1):
        for d in (64, 128):
            for rot in sorted({0, 8, 16, 22, 62, 64, d - 2, d}):
                for interleaved in (0, 1):
                    for T, n in ((1, 3), (33, 2), (300, 2), (33, 200)):
                        for block in (1, 4, 8, 16, 25, 64, 128, 255, 256):
                            got = r.append(dt=dt, d=d, rot=rot if rot else 0, interleaved=interleaved, T=T, n=n, block=block)
                            limits.setdefault(got.name, set()).add(got.allowed)
                            most[got.name] = max(most.get(got.name, 0), got.smem)
    assert all(len(x) == 1 for x in limits.values()), "a kernel's limit depends on the call"
    assert r.lib.fake_lowered() == 0
    # every instance is met, and no limit is a guess: steps of four passes are launched with all of theirs
    assert len(limits) == 2 * 2 * 4 * 5
    big = {n: (max(limits[n]), most[n]) for n in limits if most[n] > 150 << 10}
    assert big and all(allowed == used for allowed, used in big.values())


def resize(r, n, T=1, slots=True):
    """Launches of a step of n sequences and T slots each."""
    B_, t = 1 << 40, ctypes.c_void_p
    arrays = [t(B_ + i * (1 << 32)) for i in range(4)]
    return r._launched(r.lib.mha_paged_resize(arrays[0], arrays[1], n, 16, t(4096), 64, 64, t(4096), 1000, t(4096), arrays[2], arrays[3], T,
                                              t(4096) if slots else None, None))


@pytest.mark.parametrize("largest", [16, 8, 4, 2, 1])
@pytest.mark.parametrize("n", [1, 512, 513])
def test_a_resize_takes_the_largest_cluster_that_fits(linked, largest, n):
    """A part of a device, or another one, may have no room for 16 CTAs side by side: the call is then made with fewer."""
    r = Recorded(linked, f"cluster{largest}_{n}", cluster=largest)
    for _ in range(2):
        got = resize(r, n)
        assert len(got) == 1 and got[0].cluster == largest and got[0].grid[0] == largest
        assert got[0].block[0] == (512 if n <= 512 else 1024)


def test_sizes_of_grids_go_by_the_devices_sms(linked):
    """Waves and rules of as many CTAs as SMs are those of the device that runs them."""
    half, whole = Recorded(linked, "half", sms=76), Recorded(linked, "whole", sms=152)
    # fewer tiles than a wave of either: parts of the heads fill it, on both alike
    shape = dict(h=64, h_kv=64, n=4, T=64, block=32)
    a, b = half.append(**shape), whole.append(**shape)
    assert a.grid[0] == b.grid[0] and 0 < a.grid[1] < b.grid[1]
    # as many tiles as 76 SMs, but not as 152: "many" for one, and the kernel of more CTAs an SM
    shape = dict(n=50, T=64, block=4)
    a, b = half.append(**shape), whole.append(**shape)
    assert 76 <= a.grid[0] < 152 and a.grid[0] == b.grid[0] and a.name != b.name
    # the slots of many tokens
    a, b = resize(half, 64, T=1 << 16), resize(whole, 64, T=1 << 16)
    assert len(a) == len(b) == 2 and a[1].grid[0] == 8 * 76 and b[1].grid[0] == 8 * 152
