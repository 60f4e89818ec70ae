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
