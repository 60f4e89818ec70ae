"""Tensor calls of the paged key-value cache, on the host: what they refuse
before anything is launched."""
import pytest

import quantized_weight_gguf_gb300 as q
from quantized_weight_gguf_gb300 import build_lib

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    q.load()


def _cache(device):
    size = q.qmm_kv_page_bytes("q8_0", "q8_0", 16, 2, 64)
    return q.KvCache("q8_0", "q8_0", torch.zeros((3, size), dtype=torch.uint8, device=device), 16, 2, 64)


def _tensors(device):
    return dict(table=torch.tensor([[0, 2], [1, 2]], dtype=torch.int32, device=device),
                lens=torch.ones(2, dtype=torch.int32, device=device),
                x=torch.zeros((2, 1, 2, 64), device=device), to=torch.zeros((2, 1, 2, 64), device=device),
                rope=torch.zeros((8, 32, 2), device=device),
                ws=torch.zeros(1 << 20, dtype=torch.uint8, device=device))


CALLS = {
    "kv_append": lambda c, t: q.kv_append(c, t["x"], t["x"], t["table"], t["lens"], q=t["x"], q_out=t["to"],
                                          rope=t["rope"]),
    "kv_read": lambda c, t: q.kv_read(c, t["table"], t["lens"], 1, k=t["x"], v=t["to"]),
    "attend": lambda c, t: q.attend(c, t["x"], t["table"], t["lens"], out=t["to"], workspace=t["ws"]),
}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_a_pool_in_host_memory_is_refused(call):
    with pytest.raises(ValueError, match="device"):
        CALLS[call](_cache("cpu"), _tensors("cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("call,names", [("kv_append", ("table", "lens", "x", "to", "rope")),
                                        ("kv_read", ("table", "lens", "x", "to")),
                                        ("attend", ("table", "lens", "x", "to", "ws"))])
def test_tensors_in_host_memory_are_refused(call, names):
    """One tensor at a time; nothing is launched."""
    cache, here, host = _cache("cuda:0"), _tensors("cuda:0"), _tensors("cpu")
    for name in names:
        with pytest.raises(ValueError, match="device"):
            CALLS[call](cache, {**here, name: host[name]})
    CALLS[call](cache, here)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0


def test_host_threads_do_not_share_attention_scratch():
    """One call is two launches (strips, then their join), so calls of two threads can interleave on
    a stream that both use."""
    import threading

    def scratch():
        mine = [q._scratch_of_stream(n, torch.device("cpu"), 0) for n in (1000, 500, 3 << 20, 7)]
        assert mine[0] is mine[1] and mine[2] is mine[3] and mine[2].numel() >= 3 << 20
        return mine

    here, there = scratch(), []
    other = threading.Thread(target=lambda: there.extend(scratch()))
    other.start()
    other.join()
    assert len(there) == 4
    assert not {t.data_ptr() for t in here} & {t.data_ptr() for t in there}


@pytest.mark.gpu
def test_two_host_threads_on_one_stream():
    """Split items of different inputs from two threads on the default stream: every result is the
    serial one, bit for bit."""
    import threading
    torch.manual_seed(5)
    n_kv, dim, page, n = 2, 64, 16, 4000
    jobs = []
    for seed in range(2):
        per = -(-n // page)
        cache = q.KvCache.empty("q8_0", "q8_0", per, page, n_kv, dim, device="cuda:0")
        table = torch.randperm(per).to(torch.int32).view(1, per).cuda()
        lens = torch.tensor([n], dtype=torch.int32, device="cuda:0")
        k, v = torch.randn((2, 1, n, n_kv, dim), device="cuda:0")
        q.kv_append(cache, k, v, table, lens)
        x = torch.randn((1, 1, 8, dim), device="cuda:0")
        ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda:0")
        jobs.append((cache, x, table, lens, q.attend(cache, x, table, lens, workspace=ws)))
    torch.cuda.synchronize()
    start, bad = threading.Barrier(2), []

    def run(job):
        start.wait()
        for _ in range(300):
            out = q.attend(*job[:4])
            bad.append((out != job[4]).any())

    threads = [threading.Thread(target=run, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(bad) == 600 and not torch.stack(bad).any()
    assert q.qmm_device_status() == 0


def test_a_cache_keeps_its_pool():
    """The calls' arguments hold the pool's address, so another tensor cannot take its place unseen."""
    cache = _cache("cpu")
    with pytest.raises(AttributeError):
        cache.pages = torch.zeros_like(cache.pages)
    for name in ("page_size", "n_kv_heads", "head_dim"):
        with pytest.raises(AttributeError):
            setattr(cache, name, 64)
