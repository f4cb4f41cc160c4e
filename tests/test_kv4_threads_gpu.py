"""Cache calls from two host threads at a time, each on a stream of its own."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_attention_forward_b200 as lp


def _together(jobs):
    """Runs the jobs on threads of their own, started together; the first error is raised."""
    errors, gate = [], threading.Barrier(len(jobs))

    def run(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                job()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


def test_reads_of_caches_with_many_and_more_heads():
    """Each needs more than the 48 KB of shared memory that a launch has without asking, and another amount."""
    jobs, checks = [], []
    meta = lp.lpfa_varlen_meta_from_lengths([5])
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for heads in (1024, 400, 1000, 390):
        cache = lp.Kv4Cache(1, heads, 16)
        x = torch.randn(5, heads, 128, device="cuda").bfloat16()
        lp.lpfa_kv4_write(x, -x, cache, table, meta)
        want = lp.lpfa_kv4_read(cache, table, meta)
        outs = [torch.empty_like(t) for t in want]
        args = (cache._c, lp._PageTable(table.data_ptr(), 1, 1), None, meta._c, 128, *(t.data_ptr() for t in outs))

        def job(args=args):  # the library's own call: as little as possible between one and the next
            stream = torch.cuda.current_stream().cuda_stream
            for i in range(20000):
                lp._check(lp._lib.lpfa_kv4_read(*args, stream))
                if i % 500 == 499:
                    torch.cuda.current_stream().synchronize()
        jobs.append(job)
        checks.append((want, outs, cache))  # (the call has the cache's addresses alone)
    torch.cuda.synchronize()
    _together(jobs)
    for want, outs, _ in checks:
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_writes_and_attention_at_a_time():
    """Two threads append to caches of their own and attend over them; each has what it has alone."""
    def build(seed, heads, group):
        g = torch.Generator(device="cuda").manual_seed(seed)
        k, v = (torch.randn(40, heads, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        q = torch.randn(2, heads * group, 128, generator=g, device="cuda").bfloat16()
        return (k, v, q, torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3), lp.lpfa_varlen_meta_from_lengths([33, 7]),
                lp.lpfa_varlen_meta_from_lengths([1, 1]), torch.tensor([33, 7], dtype=torch.int32, device="cuda"))

    def once(k, v, q, table, meta, meta_q, lens):
        cache = lp.Kv4Cache(6, k.shape[1], 16)
        lp.lpfa_kv4_write(k, v, cache, table, meta)
        return lp.lpfa_attn_fwd_kv4(q, cache, table, lens, meta_q)

    sets = [build(1, 8, 4), build(2, 3, 1)]
    want = [once(*s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]

    def job(i):
        for _ in range(100):
            got[i] = once(*sets[i])
    _together([lambda: job(0), lambda: job(1)])
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    assert lp.lpfa_device_status() == (lp.LPFA_OK, 0)


def test_a_cache_keeps_the_tensors_that_its_calls_write_to():
    """The handle holds addresses: its tensors are its own for good, and a new pool is a new handle."""
    cache = lp.Kv4Cache(2, 1, 16)
    for name in ("k", "k_scales", "v", "v_scales"):
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros_like(getattr(cache, name)))
    same = lp.Kv4Cache.from_tensors(cache.k, cache.k_scales, cache.v, cache.v_scales)
    x = torch.randn(5, 1, 128, device="cuda").bfloat16()
    lp.lpfa_kv4_write(x, x, same, torch.ones(1, 1, dtype=torch.int32, device="cuda"), lp.lpfa_varlen_meta_from_lengths([5]))
    assert cache.k[1, 0, :5].any() and not cache.k[0].any() and torch.equal(cache.k, cache.v)
