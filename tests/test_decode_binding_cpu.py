"""What the decode binding checks of its operands' layouts, on host tensors (no GPU
needed: the device check is taken out)."""
import ctypes
import gc
import threading
import weakref

import pytest
import torch

from gemm_decode_q1_amd import decode as D
from gemm_decode_q1_amd import q1 as B


@pytest.fixture(autouse=True)
def _host(monkeypatch):
    monkeypatch.setattr(D, "_same_device", lambda first, **others: None)


def attn_layout(k_prefix, v_prefix):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    return D._check_attn(q, k_prefix, v_prefix, None, None, None, None, None, None, None)


@pytest.mark.parametrize("P", [1, 2])
@pytest.mark.parametrize("which", ["k_prefix", "v_prefix"])
@pytest.mark.parametrize("how", ["transposed", "heads expanded", "all expanded", "every second element"])
def test_prefix_must_be_dense_in_a_row(P, which, how):
    """Whatever the number of prefix tokens, keys and values of a token are dense: the kernel reads them so."""
    dense = torch.zeros(P, 2, 64, dtype=torch.bfloat16)
    odd = {"transposed": torch.zeros(P, 64, 2, dtype=torch.bfloat16).transpose(1, 2),
           "heads expanded": torch.zeros(P, 1, 64, dtype=torch.bfloat16).expand(P, 2, 64),
           "all expanded": torch.zeros(1, 1, 1, dtype=torch.bfloat16).expand(P, 2, 64),
           "every second element": torch.zeros(P, 2, 128, dtype=torch.bfloat16)[..., ::2]}[how]
    assert attn_layout(dense, dense)
    with pytest.raises(ValueError, match=which):
        attn_layout(*((odd, dense) if which == "k_prefix" else (dense, odd)))


def test_one_prefix_token_may_have_any_row_stride():
    """A single row's stride is never used: keys and values may come from differently spaced rows."""
    k, v = (torch.zeros(3, n, 64, dtype=torch.bfloat16)[:1, :2] for n in (2, 5))
    assert attn_layout(k, v)
    with pytest.raises(ValueError, match="row stride"):
        attn_layout(*(torch.zeros(3, n, 64, dtype=torch.bfloat16)[:2, :2] for n in (2, 5)))



class Library:
    """Stands in for the library: takes any call, wants 4096 bytes of workspace."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *args: 4096
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(D, "load_library", lambda: lib)
    monkeypatch.setattr(D, "_stream_of", lambda index: 0)
    monkeypatch.setattr(D, "_device", lambda: -1)
    return lib


def call(op, **kw):
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype)  # noqa: E731
    f = torch.float32
    if op == "sample":
        return D.q1_sample(z(2, 100, dtype=f), z(2, dtype=f), **kw)
    if op == "attn":
        return D.q1_prefix_attn(z(2, 4, 64), z(9, 2, 64), z(9, 2, 64), **kw)
    return D.q1_delta_prefill(z(9, 1, 64), z(9, 1, 64), z(9, 2, 64), z(9, 2, dtype=f), z(9, 2, dtype=f),
                              z(1, 2, 64, 64, dtype=f), torch.tensor([0, 9], dtype=torch.int32), **kw)


OPS = ["sample", "attn", "prefill"]


@pytest.mark.parametrize("op", OPS)
def test_a_given_workspace_is_checked(library, op):
    """Its bytes are counted from its elements, and the kernels write to all of them:
    so bytes, dense, on the operands' device."""
    call(op, workspace=torch.zeros(4096, dtype=torch.uint8))
    assert len(library.calls) == 1 and 4096 in library.calls[0][1]
    for odd in (torch.zeros(4096), torch.zeros(8192, dtype=torch.uint8)[::2],
                torch.zeros(1, dtype=torch.uint8).expand(4096)):
        with pytest.raises(ValueError, match="workspace"):
            call(op, workspace=odd)
    assert len(library.calls) == 1
    with pytest.raises(ValueError, match="workspace"):
        D._given(torch.zeros(4096, dtype=torch.uint8), 0)  # host memory beside operands on device 0


def in_thread(f):
    t = threading.Thread(target=f)
    t.start()
    t.join()


def test_a_thread_has_a_workspace_of_its_own(monkeypatch):
    """A call is several launches that hand data on through its workspace, and another thread's may come
    between them on the same stream: threads share none.  A thread's calls share one, freed as it ends."""
    made = []

    def empty(n, dtype, device):
        t = torch.empty(n, dtype=dtype)
        made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(D, "_empty", empty)
    monkeypatch.setattr(D, "_capturing", lambda: False)

    def nested():
        mine = D._workspace(100000, 0, 7)
        assert D._workspace(4096, 0, 7) is mine and D._workspace(4096, 0, 8) is not mine
        in_thread(lambda: others.append(D._workspace(4096, 0, 7)))
        assert others and others[0] is not mine and others[0].data_ptr() != mine.data_ptr()
        done.append(1)

    others, done = [], []
    in_thread(nested)
    assert done and len(made) == 3
    others.clear()
    gc.collect()
    assert all(r() is None for r in made)


def test_a_large_workspace_is_not_kept(monkeypatch):
    monkeypatch.setattr(D, "_empty", lambda n, dtype, device: torch.empty(n, dtype=dtype))
    monkeypatch.setattr(D, "_capturing", lambda: False)
    D._workspace(4096, 0, 9)
    large = weakref.ref(D._workspace(264 << 20, 0, 9))
    gc.collect()
    assert large() is None and D._scratch.kept.pop((0, 9)).numel() < 1 << 20


def test_packed_calls_share_no_workspace_between_threads(monkeypatch):
    monkeypatch.setattr(B, "_stream", lambda device=None: ctypes.c_void_p(7))
    spaces, host, got = B._Workspaces(), torch.device("cpu"), []
    take = lambda: got.append(spaces.get(1000, host))  # noqa: E731
    take()
    in_thread(take)
    take()
    assert got[0] is got[2] and got[1] is not got[0] and got[0].data_ptr() != got[1].data_ptr()
