"""linear8 under torch.autograd: what it keeps for its backward pass, and for how long.

The kernels' places are taken by plain products on the CPU; inputs are small whole numbers,
which e4m3 holds, so that every result is exact.
"""
import numpy as np
import pytest

from matrix_orthogonalising_optimizer_02_amd import blocks8
import matrix_orthogonalising_optimizer_02_amd as muon

torch = pytest.importorskip("torch")


class Recorder:
    """quantise8 and matmul8 on the CPU, all powers 1, and a note of each call."""

    def __init__(self):
        self.made, self.forms, self.products = [], [], []

    def quantise8(self, x, *, tiles=False, direct=True, transposed=False, out=None, out_transposed=None, stream=None):
        flat = x.detach().reshape(-1, x.shape[-1])
        self.forms.append((tuple(flat.shape), direct or out is not None, transposed or out_transposed is not None))
        q = self.one(flat, tiles, out) if direct or out is not None else None
        qt = self.one(flat.t(), tiles, out_transposed) if transposed or out_transposed is not None else None
        return q, qt

    def one(self, m, tiles, out):
        q = blocks8._new(torch.empty(0), m.shape[0], m.shape[1], tiles) if out is None else out
        q.codes.copy_(torch.nn.functional.pad(m.float(), (0, q.codes.shape[1] - m.shape[1])).to(torch.float8_e4m3fn))
        q.scales.fill_(127)
        self.made.append(q)
        return q

    def matmul8(self, a, b, *, dtype=None, products=None, **kw):
        assert a.cols == b.cols and a.codes.shape[0] == a.rows and b.codes.shape[0] == b.rows
        assert a.tiles is False
        self.products.append(products)
        return (a.codes.float()[:, :a.cols] @ b.codes.float()[:, :b.cols].t()).to(dtype)


@pytest.fixture
def fake(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(blocks8, "quantise8", r.quantise8)
    monkeypatch.setattr(blocks8, "matmul8", r.matmul8)
    return r


def whole(seed, *shape, grad=True):
    gen = np.random.default_rng(seed)
    return torch.from_numpy(gen.integers(-3, 4, shape).astype(np.float32)).requires_grad_(grad)


def storages(quantised):
    from torch.multiprocessing.reductions import StorageWeakRef
    return [StorageWeakRef(t.untyped_storage()) for q in quantised for t in (q.codes, q.scales)]


@pytest.mark.parametrize("kept", [False, True])
def test_gradients(fake, kept):
    x, w, g = whole(1, 2, 5, 7), whole(2, 6, 7), whole(3, 2, 5, 6, grad=False)
    muon.linear8(x, w, muon.Weight8(w) if kept else None).backward(g)
    assert torch.equal(x.grad, g @ w.detach()) and torch.equal(w.grad, g.reshape(-1, 6).t() @ x.detach().reshape(-1, 7))


def test_operands_go_with_the_backward_pass(fake):
    """The output lives on; what the backward pass read does not."""
    x, w, g = whole(1, 5, 7), whole(2, 6, 7), whole(3, 5, 6, grad=False)
    y = muon.linear8(x, w)
    held = storages(fake.made)
    fake.made.clear()
    assert sum(not s.expired() for s in held) == 4  # the transposed x and weight
    y.backward(g)
    fake.made.clear()
    assert all(s.expired() for s in held)


@pytest.mark.parametrize("kept", [False, True])
def test_a_second_backward_pass_is_refused(fake, kept):
    x, w, g = whole(1, 5, 7), whole(2, 6, 7), whole(3, 5, 6, grad=False)
    y = muon.linear8(x, w, muon.Weight8(w) if kept else None)
    y.backward(g, retain_graph=True)
    y.backward(g)
    assert torch.equal(w.grad, 2 * (g.t() @ x.detach()))
    with pytest.raises(RuntimeError, match="second time"):
        y.backward(g)


def test_hooks_see_what_is_kept(fake):
    """saved_tensors_hooks get the 8-bit operands, and the backward pass takes what they give back."""
    x, w, g = whole(1, 5, 7), whole(2, 6, 7), whole(3, 5, 6, grad=False)
    packed, unpacked = [], []

    def pack(t):
        packed.append(t.dtype)
        return t.clone()

    def unpack(t):
        unpacked.append(t.dtype)
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
        y = muon.linear8(x, w)
    held = storages(fake.made)
    fake.made.clear()
    assert all(s.expired() for s in held)  # the clones alone are kept
    y.backward(g)
    assert sorted(map(str, packed)) == sorted(map(str, unpacked)) == ["torch.float8_e4m3fn"] * 2 + ["torch.uint8"] * 2
    assert torch.equal(x.grad, g @ w.detach()) and torch.equal(w.grad, g.t() @ x.detach())


def test_checkpointing_keeps_no_operand(fake):
    x, w, g = whole(1, 5, 7), whole(2, 6, 7), whole(3, 5, 6, grad=False)
    y = torch.utils.checkpoint.checkpoint(lambda a, b: muon.linear8(a, b), x, w, use_reentrant=False)
    held = storages(fake.made)
    fake.made.clear()
    assert all(s.expired() for s in held)
    y.backward(g)
    assert torch.equal(x.grad, g @ w.detach()) and torch.equal(w.grad, g.t() @ x.detach())


def test_a_form_that_moved_on_is_refused(fake):
    x, w, g = whole(1, 5, 7), whole(2, 6, 7), whole(3, 5, 6, grad=False)
    w8 = muon.Weight8(w)
    y = muon.linear8(x, w, w8)
    w8.update(w)
    with pytest.raises(RuntimeError, match="updated after"):
        y.backward(g)


@pytest.mark.parametrize("grads", ["no_grad", "inference", "frozen"])
def test_no_form_that_no_gradient_reads(fake, grads):
    """Without gradients x and the weight are quantised in the form that the output reads alone."""
    frozen = grads == "frozen"
    x, w = whole(1, 5, 7, grad=not frozen), whole(2, 6, 7, grad=not frozen)
    with {"no_grad": torch.no_grad, "inference": torch.inference_mode, "frozen": torch.enable_grad}[grads]():
        y = muon.linear8(x, w)
    assert not y.requires_grad and torch.equal(y, x.detach() @ w.detach().t())
    assert sorted(fake.forms) == [((5, 7), True, False), ((6, 7), True, False)]


def test_forms_of_one_gradient(fake):
    x, w, g = whole(1, 5, 7), whole(2, 6, 7), whole(3, 5, 6, grad=False)
    muon.linear8(x, w.detach()).backward(g)
    assert sorted(fake.forms) == [((5, 6), True, False), ((5, 7), True, False), ((6, 7), True, True)]
    fake.forms.clear()
    muon.linear8(x.detach(), w).backward(g)
    assert sorted(fake.forms) == [((5, 6), False, True), ((5, 7), True, True), ((6, 7), True, False)]
    assert torch.equal(x.grad, g @ w.detach()) and torch.equal(w.grad, g.t() @ x.detach())


def test_refused_at_the_call(fake):
    """What the backward pass could not do is refused by the forward call."""
    x, w = whole(1, 5, 8), whole(2, 6, 8)
    w8 = muon.Weight8(w)
    for call, text in ((lambda: muon.linear8(x, w.detach().double().requires_grad_(), w8), "weight must be float32"),
                       (lambda: muon.linear8(x, w.detach().double()), "weight must be float32"),
                       (lambda: muon.linear8(x.detach().double(), w, w8), "x must be float32"),
                       (lambda: muon.linear8(x, w.detach().to("meta").requires_grad_(), w8), "weight must live on cpu"),
                       (lambda: muon.linear8(x, w.detach().to("meta")), "weight must live on cpu"),
                       (lambda: muon.linear8(x, w, w8, weight_grad_products=4), "products must be None, 8 or 16")):
        fake.forms.clear()
        with pytest.raises(ValueError, match=text):
            call()
        assert not fake.forms


def test_products_of_each_result(fake):
    x, w, g = whole(1, 5, 7), whole(2, 6, 7), whole(3, 5, 6, grad=False)
    for more, want in (({}, [None, None, None]), (dict(products=16), [16, 16, None]), (dict(products=8, weight_grad_products=16), [8, 8, 16]),
                       (dict(weight_grad_products=8), [None, None, 8])):
        fake.products.clear()
        muon.linear8(x, w, **more).backward(g)
        assert fake.products == want
    with pytest.raises(ValueError, match="products must be None, 8 or 16"):
        muon.linear8(x, w, products=0)


def test_a_weight_that_is_its_8_bit_form_alone(fake):
    """With a kept form and no gradient of its own, a weight lends its shape: the full one may be
    elsewhere, in any type, or nowhere."""
    x, w, g = whole(1, 5, 7), whole(2, 6, 7, grad=False), whole(3, 5, 6, grad=False)
    w8 = muon.Weight8(w)
    for other in (w.to("meta"), w.double()):
        x.grad = None
        muon.linear8(x, other, w8).backward(g)
        assert torch.equal(x.grad, g @ w)
    with torch.no_grad():
        assert torch.equal(muon.linear8(x, w.to("meta").requires_grad_(), w8), x @ w.t())
