"""The operators around a cache in 8 bits on the GPU: calls from several host threads."""
import threading

import pytest

torch = pytest.importorskip("torch")

from test_coded_gpu import BF, E4, bnd, clean_status, freqs, ints, pages_of, randn, same, table_of  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ append
def test_appends_from_two_host_threads(bnd):
    """Blocks of 64 and of 256 tokens through one kernel, which need different amounts of shared memory, call after call from
    two host threads at once: every call is taken, with the results of calls one after the other."""
    h, hk, d, T = 4, 2, 128, 256
    jobs = []
    for i, block in enumerate((64, 256)):
        table, n_pages = table_of(i, 2, 2)
        kp, ks = pages_of(6 + i, n_pages, 256, block, hk, d, E4)
        vp, vs = pages_of(8 + i, n_pages, 256, block, hk, d, E4)
        q, k, v = (randn(10 + i + 3 * j, 2, T, (h, hk, hk)[j], d, dtype=BF) for j in range(3))
        cache, rotary = bnd.make_coded_cache(kp, vp, ks, vs, table), bnd.make_rotary(freqs(128 if block == 256 else 16))
        start, out = ints([0, 256]), torch.zeros_like(q)
        outs = (kp, vp, ks, vs, out)

        def call(stream=None, a=(k, v, start), kw=dict(cache=cache, q=q, q_out=out, rotary=rotary)):
            bnd.mha_coded_append(*a, stream=stream, **kw)

        def clear(cleared=(kp, vp, out)):        # pages that no call writes are zeros before and after
            for o in cleared:
                o.view(torch.uint8).zero_()
        clear()
        call()
        torch.cuda.synchronize()
        jobs.append((call, outs, [o.clone() for o in outs], torch.cuda.Stream()))
        clear()
    torch.cuda.synchronize()
    errors, begin = [], threading.Barrier(2)

    def work(call, stream):
        try:
            begin.wait(30)
            for _ in range(3000):
                call(stream)
            stream.synchronize()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j[0], j[3])) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for _, outs, want, _ in jobs:
        assert all(same(a, b) for a, b in zip(outs, want))
