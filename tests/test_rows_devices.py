"""Calls on rows of scores check every tensor they hand to a kernel, those behind a handle too:
all on the current device, whose streams the launch goes to. On the CPU, with tensors that
claim a device and a library that must not be reached."""
import pytest
import torch

import sparse_embedding_exact_amd as sps


class On(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True
    gpu = 0

    def get_device(self):
        return self.gpu


def on(gpu, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.gpu = gpu
    return t


def csr(indptr=0, indices=0, values=0):
    return sps.CSR(on(indptr, 4, dtype=torch.int32), on(indices, 6, dtype=torch.int32), on(values, 6),
                   3, 9)


class Reached(Exception):
    pass


class Library:
    def __getattr__(self, name):
        if name.endswith("_destroy"):
            return lambda h: None
        if name.endswith("_size"):
            return lambda *a: 0

        def reached(*a):
            raise Reached(name)
        return reached


@pytest.fixture
def calls(monkeypatch):
    monkeypatch.setattr(sps, "_lib", Library())
    monkeypatch.setattr(sps, "_stream_of", lambda device, stream: 0)
    monkeypatch.setattr(sps, "_stream_ptr", lambda stream=None: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    sps._sized.cache_clear()
    yield
    sps._sized.cache_clear()


def handle(gpu):
    return sps.Distill(None, on(gpu, 64, dtype=torch.uint8), 3, 5, "cpu")


def items(gpu):
    it = object.__new__(sps.Items)
    it._h, it._persistent = None, on(gpu, 64, dtype=torch.uint8)
    return it


def i32(gpu, *shape):
    return on(gpu, *shape, dtype=torch.int32)


GRAD = dict(
    chunk_rows=lambda a, b, c, o, g, d: sps.cosine_chunk_grad(csr(a, b, c), items(o), 0, on(g, 3, 5), on(d, 6)),
    values=lambda a, b, c, o, g, d: sps.cosine_grad_values(csr(a, b, c), on(g, 6), on(d, 6)),
    queries=lambda a, b, c, o, g, d: sps.cosine_grad(csr(a, b, c), csr(o, g, d), on(0, 3, 3)),
    both=lambda a, b, c, o, g, d: sps.bulk_distill(csr(a, b, c), csr(o, g, d), i32(0, 3, 2), on(0, 3, 2)),
    select=lambda a, b, c, o, g, d: sps.bulk_select(csr(a, b, c), csr(o, g, d), 4),
)
# cosine_grad_values has no other side
WHICH = [(c, w) for c in GRAD for w in (None, 0, 1, 2, 3, 4, 5) if (c, w) != ("values", 3)]


@pytest.mark.parametrize("call,which", WHICH)
def test_gradient_of_scores(calls, call, which):
    gpus = [1 if i == which else 0 for i in range(6)]
    with pytest.raises(Reached if which is None else AssertionError):
        GRAD[call](*gpus)


@pytest.mark.parametrize("h,x", [(0, 0), (1, 0), (0, 1)])
def test_distillation_handles(calls, h, x):
    want = Reached if (h, x) == (0, 0) else AssertionError
    with pytest.raises(want):
        sps.distill_chunk(handle(h), on(x, 3, 5), first=True)
    with pytest.raises(want):
        sps.distill_chunk_grad(handle(h), on(x, 3, 5), out=on(x, 3, 5))


@pytest.mark.parametrize("ids,t,w", [(1, 0, 0), (0, 1, 0), (0, 0, 1)])
def test_bulk_distill_lists(calls, ids, t, w):
    with pytest.raises(AssertionError):
        sps.bulk_distill(csr(), csr(), i32(ids, 3, 2), on(t, 3, 2), row_weights=on(w, 3))
