"""What the binding allocates for a call on another stream comes from that
stream's pool (a block of the current stream's may still be in use by work
queued there), shown with a stand-in for the library and the allocator."""
import contextlib
import types

import pytest
import torch

import attention_split_attn_b200 as A

HERE, SIDE = "current stream", types.SimpleNamespace(cuda_stream=7)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def record_stream(self, s):
        OnGpu.recorded.append((self.data_ptr(), s))


@pytest.fixture
def gpu(monkeypatch):
    """The calls made (name, stream handle) and the allocations (address, stream)."""
    log = types.SimpleNamespace(calls=[], allocated=[], recorded=[], current=HERE)
    OnGpu.recorded = log.recorded

    @contextlib.contextmanager
    def stream(s):
        before, log.current = log.current, s
        yield
        log.current = before

    real_empty = torch.empty

    def empty(*shape, dtype=None, device=None):
        t = real_empty(*shape, dtype=dtype).as_subclass(OnGpu)
        log.allocated.append((t.data_ptr(), log.current))
        return t

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *a: 4096
            if name.endswith("supports"):
                return lambda *a: 0
            handle = -2 if name.endswith("_timed") else -1
            return lambda *a: log.calls.append((name, a[handle])) or 0

    monkeypatch.setattr(A, "load_library", Lib)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: HERE)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return log


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32).as_subclass(OnGpu)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16).as_subclass(OnGpu)


def _paged():
    q, k = _bf16(2, 4, 64), _bf16(3, 16, 2, 64)
    return A.make_paged_args(q, k, k, q, _i32(0, 1).view(2, 1), _i32(5, 5), scale=1.0)


def _flat():
    q, k = _bf16(2, 4, 64), _bf16(16, 2, 64)
    return A.make_args(q, k, k, q, scale=1.0)


CALLS = {
    "decode_paged": lambda s: A.attn_decode_paged_args(_paged(), stream=s),
    "decode_shared": lambda s: A.attn_decode_shared_args(_paged(), stream=s),
    "decode": lambda s: A.attn_decode_args(_flat(), stream=s),
    "decode_append": lambda s: A.attn_decode_append_args(_flat(), _bf16(2, 2, 64), _bf16(2, 2, 64), stream=s),
    "prefill": lambda s: A.attn_prefill_args(_flat(), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_workspace_belongs_to_the_stream_of_the_call(gpu, name):
    ws = CALLS[name](SIDE)
    assert gpu.calls == [("attn_" + name, 7)]
    assert gpu.allocated == [(ws.data_ptr(), SIDE)]


@pytest.mark.parametrize("given", [False, True])
def test_page_tables_belong_to_the_stream_of_the_call(gpu, given):
    out = A.PageTables(*(_i32(*[0] * 9) for _ in A.PageTables._fields)) if given else None
    o = A.page_tables(_i32(0, 0), _i32(1, 1), _i32(0, 0, 0, 0).view(2, 2), _i32(1, 2, 3), _i32(0, 3), page_size=16,
                      n_rows=4, outputs=out, stream=SIDE)
    assert gpu.calls == [("attn_page_tables", 7)]
    new = [] if given else [t.data_ptr() for t in o]
    assert gpu.allocated == [(p, SIDE) for p in new]
    assert gpu.recorded == [(p, HERE) for p in new]     # and the caller reads them on the current stream


def test_tree_mask_belongs_to_the_stream_of_the_call(gpu):
    m = A.tree_mask(_i32(-1, 0), 3, 8, stream=SIDE)
    assert gpu.calls == [("attn_tree_mask", 7)]
    assert gpu.allocated == [(m.data_ptr(), SIDE)] and gpu.recorded == [(m.data_ptr(), HERE)]


def test_allocations_without_a_stream_stay_on_the_current_one(gpu, monkeypatch):
    monkeypatch.setattr(A, "_raw_stream", lambda dev: 1)
    ws = A.attn_decode_paged_args(_paged())
    assert gpu.allocated == [(ws.data_ptr(), HERE)] and not gpu.recorded
