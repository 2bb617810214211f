"""The fine-tuning example on MI355X: the operators together, as a user runs them."""
import importlib.util
import os

import pytest

from gpu_util import log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "finetune_adapters.py")


def load():
    spec = importlib.util.spec_from_file_location("finetune_adapters", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_adapters_learn_and_serve():
    log("example")
    losses, _ = load().main(steps=60)
    assert losses.isfinite().all()
    # it starts at the entropy of a guess (log 1000 = 6.9, the random head adds
    # about 1) and has to have learned something of both tasks
    assert losses[-5:].mean() < losses[:5].mean() - 0.3


def test_gradients_of_the_whole_model():
    # one step's parameter changes against float32 autograd of the same model on the
    # same bf16 parameters: the activations and gradients between the operators
    # are rounded to bf16 (2^-8 a rounding, about a dozen of them in a row), so the
    # gradients agree to a few percent in norm
    log("example gradients")
    ex = load()
    model = ex.Model()
    follow = ex.tasks()
    tokens, adapter, labels = ex.batch(follow, 5)
    for i in range(ex.LAYERS):
        model.params[f"B{i}"] += 0.02 * torch.randn_like(model.params[f"B{i}"])
    p = {k: v.float().requires_grad_() for k, v in model.rounded().items()}
    x = model.embedding[tokens].float()
    norm = lambda t, w, b: torch.nn.functional.layer_norm(t, (ex.WIDTH,), w, b)
    for i, (values, idx) in enumerate(model.packed):
        W = ex.nm.nm_decompress(values, idx, ex.WIDTH).float()
        h = norm(x, p[f"norm{i}"], p[f"norm{i}_bias"])
        y = h @ W.t()
        for a in range(2):
            at = (adapter == a).float()[:, None]
            y = y + at * model.scale[a] * (h @ p[f"A{i}"][a].t() @ p[f"B{i}"][a].t())
        x = x + y
    logits = norm(x, p["norm"], p["norm_bias"]) @ p["head"].t()
    loss = torch.nn.functional.cross_entropy(logits, labels.long(), ignore_index=-100)
    loss.backward()
    before = {k: v.clone() for k, v in model.params.items()}
    got = model.step(tokens, adapter, labels, 1.0)
    torch.cuda.synchronize()
    assert abs(got.item() - loss.item()) < 0.02 * loss.item()
    for k in before:
        g, r = before[k] - model.params[k], p[k].grad
        err = ((g - r).norm() / r.norm()).item()
        assert err < 0.05, (k, err)


def test_captured_in_a_graph():
    # the serving path (norm, few-token adapter product) and the loss with its gradient,
    # captured once and replayed on new inputs, with eager work in between
    log("example graph")
    ex = load()
    nm = ex.nm
    model = ex.Model()
    p = model.rounded()
    p["B0"] = torch.randn_like(p["B0"])
    values, idx = model.packed[0]

    def work(x, ids, labels, weight):
        h, mean, rstd = nm.nm_layernorm(x, p["norm0"], p["norm0_bias"], stats=True)
        y, xa = nm.nm_adapter_spmm(values, idx, h, ids, p["A0"], p["B0"], model.scale, ex.WIDTH)
        loss, lse = nm.nm_xent(h, p["head"], labels)
        d, dw = nm.nm_xent_bwd(h, p["head"], labels, lse, weight, out_dtype=ex.BF16)
        dh, dA, dB = nm.nm_adapter_spmm_bwd(values, idx, d, h, xa, ids, p["A0"], p["B0"], model.scale, ex.WIDTH)
        dx, dg, db = nm.nm_layernorm_bwd(d, x, mean, rstd, p["norm0"])
        return [y, xa, loss, lse, dw, dh, dA, dB, dx, dg, db]

    for T in (4, 300):
        fresh = lambda seed: (torch.randn(T, ex.WIDTH, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(ex.BF16),
                              (torch.arange(T, device="cuda") * 3 // T - 1).to(torch.int32),
                              ((torch.arange(T, device="cuda") * 37 + seed) % ex.VOCAB).to(torch.int32),
                              torch.full((T,), 1.0 / T, device="cuda"))
        held = fresh(0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work(*held)                   # first calls, outside the capture
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = work(*held)
        for seed in (1, 2, 3, 4):
            new = fresh(seed)
            ref = work(*new)
            torch.cuda.synchronize()
            for a, b in zip(held, new):
                a.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))
