"""Argument checks of the token embedding and of the gradients' norm and
clipping: refused on the host, before any launch.  No GPU is needed; the
addresses are never followed."""
import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import _binding as B

NULL, SIZE, ALIGN, ARG = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from bit_blockwise_adamw_gb300 import build
    build.build()
    return q8.load_library()


def test_every_entry_point_is_in_the_package():
    names = [n for n in q8.EXPORTS if n.startswith(("q8_embedding", "q8_grad", "q8_clip"))]
    assert len(names) == 6 and all(callable(getattr(q8, n, None)) for n in names) and callable(q8.pack_grads)


def embedding(**kw):
    base = dict(ids=0x10000, tokens=8, vocab=100, dim=64, dtype=0, scale=1.0)
    base.update(kw)
    return B._EMBEDDING.pack(*[v or 0 for v in base.values()])


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), NULL), (dict(ids=0x10004), ALIGN), (dict(tokens=-1), SIZE), (dict(tokens=1 << 30), SIZE),
    (dict(vocab=0), SIZE), (dict(vocab=1 << 31), SIZE), (dict(dim=0), SIZE), (dict(dim=1 << 30), SIZE), (dict(dtype=2), ARG),
    (dict(dtype=-1), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG)])
def test_embedding_refuses(lib, kw, code):
    e = embedding(**kw)
    assert lib.q8_embedding_forward(e, 0x20000, 0x30000, 64, None) == code
    assert lib.q8_embedding_backward(e, 0x30000, 64, 0x20000, 0, 0x40000, 1 << 40, None) == code
    assert lib.q8_embedding_workspace(e) == code
    assert q8.q8_last_error()


def test_embedding_refuses_its_other_arguments(lib):
    e, f = embedding(), embedding(dtype=1)
    forward = lambda e=e, table=0x20000, out=0x30000, stride=64: lib.q8_embedding_forward(e, table, out, stride, None)
    assert forward(e=None) == NULL
    assert forward(table=None) == NULL
    assert forward(table=0x20001) == ALIGN
    assert forward(out=None) == NULL
    assert forward(out=0x30001) == ALIGN
    assert forward(e=f, out=0x30002) == ALIGN
    assert forward(stride=63) == SIZE
    back = lambda e=e, dout=0x30000, stride=64, dtable=0x20000, acc=0, ws=0x40000, size=1 << 40: \
        lib.q8_embedding_backward(e, dout, stride, dtable, acc, ws, size, None)
    assert back(e=None) == NULL
    assert back(dout=None) == NULL
    assert back(dout=0x30001) == ALIGN
    assert back(e=f, dout=0x30002) == ALIGN
    assert back(stride=63) == SIZE
    assert back(dtable=None) == NULL
    assert back(dtable=0x20001) == ALIGN
    assert back(acc=2) == ARG
    assert back(acc=-1) == ARG
    many = embedding(tokens=5000)
    need = lib.q8_embedding_workspace(many)
    assert need > 0
    assert back(e=many, ws=None) == NULL
    assert back(e=many, ws=0x40010) == ALIGN
    assert back(e=many, size=need - 1) == SIZE
    # no tokens: nothing is launched
    assert forward(e=embedding(tokens=0, ids=None), out=None, stride=0) == 0
    assert back(e=embedding(tokens=0, ids=None), dout=None, acc=1) == 0


def grad(**kw):
    base = dict(grad=0x10000, out=0x10000, numel=1000, grad_dtype=0, out_dtype=0)
    base.update(kw)
    return B._GRAD.pack(*[v or 0 for v in base.values()])


@pytest.mark.parametrize("kw,norm_code,clip_code", [
    (dict(grad=None), NULL, NULL), (dict(grad=0x10001, out=0x20000), ALIGN, ALIGN),
    (dict(grad=0x10002, grad_dtype=1, out=0x20000), ALIGN, ALIGN), (dict(numel=-1), SIZE, SIZE), (dict(numel=1 << 40), SIZE, SIZE),
    (dict(grad_dtype=2), ARG, ARG), (dict(out=None), None, NULL), (dict(out=0x20001), None, ALIGN),
    (dict(out=0x20002, out_dtype=1), None, ALIGN), (dict(out_dtype=-1), None, ARG), (dict(out_dtype=1), None, ARG),
    (dict(grad_dtype=1), None, ARG)])
def test_grads_refuse(lib, kw, norm_code, clip_code):
    two = grad() + grad(**kw)
    if norm_code is not None:
        assert lib.q8_grad_norm(two, 2, 0x30000, 0x40000, 1 << 40, None) == norm_code
        assert "gradient 1" in q8.q8_last_error()
    assert lib.q8_clip_grads(two, 2, 1.0, 0x30000, 0x40000, 1 << 40, None) == clip_code
    assert "gradient 1" in q8.q8_last_error()


def test_grads_refuse_their_other_arguments(lib):
    need = lib.q8_grad_norm_workspace(1)
    assert need > 0 and lib.q8_grad_norm_workspace(-1) == SIZE
    norm = lambda g=grad(), n=1, norm=0x30000, ws=0x40000, size=1 << 40: lib.q8_grad_norm(g, n, norm, ws, size, None)
    clip = lambda g=grad(), n=1, limit=1.0, norm=0x30000, ws=0x40000, size=1 << 40: \
        lib.q8_clip_grads(g, n, limit, norm, ws, size, None)
    for call in (norm, clip):
        assert call(g=None) == NULL
        assert call(n=-1) == SIZE
        assert call(norm=None) == NULL
        assert call(norm=0x30002) == ALIGN
        assert call(ws=None) == NULL
        assert call(ws=0x40008) == ALIGN
        assert call(size=need - 1) == SIZE
    assert clip(limit=-1.0) == ARG
    assert clip(limit=float("nan")) == ARG


def test_binding_refuses_host_tensors_and_mismatches(lib):
    ids, w, out = torch.zeros(2, dtype=torch.int64), torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="table must be"):
        q8.q8_embedding_forward(ids, w, out)
    with pytest.raises(ValueError, match="dtable must be"):
        q8.q8_embedding_backward(ids, out, w)
    with pytest.raises(ValueError, match="dtable must be"):
        q8.q8_embedding_workspace(ids, out, w[0])
    with pytest.raises(ValueError, match="CUDA tensors"):
        q8.pack_grads([w])
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        q8.pack_grads([w.half()])
    for bad in (w.t(), w.float().to_sparse(), torch.zeros(6, device="meta")[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            q8.pack_grads([bad])
    with pytest.raises(ValueError, match="CUDA tensors"):
        q8.pack_grads([torch.zeros(6, device="meta")])
    with pytest.raises(ValueError, match="must be tensors"):
        q8.pack_grads([None])
    with pytest.raises(ValueError, match="number of elements"):
        q8.pack_grads([w], [])
    with pytest.raises(TypeError):
        q8.pack_grads(3)
    assert q8.pack_grads([]).count == 0 and q8.pack_grads(iter([])).bytes == b""
    with pytest.raises(ValueError, match="norm must be"):
        q8.q8_grad_norm([], torch.zeros(1))
