"""One training step of a mixture-of-experts block over the virtual ranks of one GPU.

Every rank holds its own tokens, one expert of each layer and a copy of the norms'
weights.  Forward: the norm after the previous block with the residual and the norm
before this one (block_norm), tokens sorted to experts (expert_sort) and copied to equal
blocks (expert_dispatch), the AlltoAll, the expert's two products (block_linear), the
AlltoAll back, the weighted sum per token (expert_combine) onto the stream.  Backward:
the same way in reverse, and the norms' gradients summed over the ranks (AllReduce).

    python examples/expert_block.py [--ranks 4] [--tokens 512] [--hidden 1024] [--inner 2048]

prints how far the step is from a plain computation in 64 bits, and its time.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_allreduce_amd as rr  # noqa: E402

CHOICES = 2
EPS = 1e-6


def make(ranks, tokens, hidden, inner, seed=0, device="cuda"):
    """The inputs and weights of every rank, bf16."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=device) * scale).bfloat16()

    each = [dict(x=rnd(tokens, hidden), branch=rnd(tokens, hidden), dout=rnd(tokens, hidden),
                 w1=rnd(inner, hidden, scale=hidden ** -0.5), b1=rnd(inner, scale=0.1),
                 w2=rnd(hidden, inner, scale=inner ** -0.5), b2=rnd(hidden, scale=0.1),
                 router=rnd(ranks, hidden, scale=hidden ** -0.5)) for _ in range(ranks)]
    post, pre = 1 + rnd(hidden, scale=0.1), 1 + rnd(hidden, scale=0.1)
    for r in each:
        r.update(post=post, pre=pre, router=each[0]["router"])
    return each


def route(y, router):
    """Each token's experts and their weights (fp32), from the router's logits."""
    logits = rr.block_linear(y, router).float()
    top = torch.topk(logits, CHOICES, dim=1)
    return top.indices, torch.softmax(top.values, 1)


def step(each, capacity):
    """Forward and backward of all ranks; adds the results to each rank's dict.  The
    routing weights' gradient ends at the weights (dweights)."""
    ranks = len(each)
    norm = dict(eps=EPS)
    for r in each:
        r["h"], r["y"] = rr.block_norm(r["x"], r["branch"], post_weight=r["post"],
                                       pre_weight=r["pre"], **norm)
        r["ids"], r["weights"] = route(r["y"], r["router"])
        r["order"] = rr.expert_sort(r["ids"], ranks, capacity)
        r["sent"] = rr.expert_dispatch(r["y"], r["order"].slots, r["order"].sources)
    for r, rows in zip(each, rr.alltoall([r["sent"] for r in each])):
        r["rows"] = rows
        r["mid"], r["z1"] = rr.block_linear(rows, r["w1"], r["b1"], act="silu", save_preact=True)
        r["made"] = rr.block_linear(r["mid"], r["w2"], r["b2"])
    for r, back in zip(each, rr.alltoall([r["made"] for r in each])):
        r["back"] = back
        r["out"] = rr.expert_combine(back, r["order"].slots, r["weights"])
    # backward; dout is the gradient by out and by the stream h that out is added to
    for r in each:
        o = r["order"]
        r["dback"], r["dweights"] = rr.expert_combine_backward(r["dout"], r["back"], o.slots,
                                                               o.sources, r["weights"])
    for r, dmade in zip(each, rr.alltoall([r["dback"] for r in each])):
        second = rr.block_linear_backward(dmade, r["mid"], r["w2"])
        first = rr.block_linear_backward(second.dx, r["rows"], r["w1"], r["z1"], act="silu")
        r.update(dw2=second.dw, db2=second.db, dw1=first.dw, db1=first.db, drows=first.dx)
    for r, dsent in zip(each, rr.alltoall([r["drows"] for r in each])):
        dy = rr.expert_dispatch_backward(dsent, r["order"].slots)
        d = rr.block_norm_backward(r["dout"], dy, r["h"], r["branch"], post_weight=r["post"],
                                   pre_weight=r["pre"], **norm)
        r.update(dx=d.dx, dbranch=d.dbranch, dpost=d.dpost_weight, dpre=d.dpre_weight)
    rr.allreduce_ring([r["dpost"] for r in each])
    rr.allreduce_ring([r["dpre"] for r in each])
    return each


def plain(each, capacity):
    """The same step in 64 bits by torch's autograd, with the routing taken from ``step``."""
    names = ("x", "branch", "w1", "b1", "w2", "b2", "weights")
    leaf = [{k: r[k].double().requires_grad_() for k in names} for r in each]
    shared = {k: each[0][k].double().requires_grad_() for k in ("post", "pre")}
    outs, loss = [], 0.0

    def unit(v):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)

    for r, p in zip(each, leaf):
        h = p["x"] + unit(p["branch"]) * shared["post"]
        y = unit(h) * shared["pre"]
        out = torch.zeros_like(y)
        for e, q in enumerate(leaf):
            t, j = torch.nonzero(r["ids"] == e, as_tuple=True)
            t, j = t[:capacity], j[:capacity]        # pairs in order; later ones are dropped
            z = y[t] @ q["w1"].t() + q["b1"]
            made = (z * torch.sigmoid(z)) @ q["w2"].t() + q["b2"]
            out = out.index_add(0, t, made * p["weights"][t, j][:, None])
        outs.append(out)
        loss = loss + ((out + h) * r["dout"].double()).sum()
    loss.backward()
    return outs, leaf, shared


def errors(each, capacity):
    """Relative distance (2-norms) of each result from the plain step's, the worst rank's."""
    outs, leaf, shared = plain(each, capacity)

    def off(a, b):
        return float((a.double() - b.detach()).norm() / b.detach().norm())

    far = {"out": max(off(r["out"], o) for r, o in zip(each, outs))}
    for name in ("x", "branch", "w1", "b1", "w2", "b2", "weights"):
        far["d" + name] = max(off(r["d" + name], p[name].grad) for r, p in zip(each, leaf))
    for name in ("post", "pre"):
        far["d" + name] = max(off(r["d" + name], shared[name].grad) for r in each)
    return far


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--ranks", type=int, default=4)
    a.add_argument("--tokens", type=int, default=512)
    a.add_argument("--hidden", type=int, default=1024)
    a.add_argument("--inner", type=int, default=2048)
    a = a.parse_args(argv)
    capacity = (a.tokens * CHOICES * 5 // 4 + a.ranks - 1) // a.ranks
    each = step(make(a.ranks, a.tokens, a.hidden, a.inner), capacity)
    far = errors(each, capacity)
    print("off by " + ", ".join(f"{k} {v:.1e}" for k, v in far.items()), flush=True)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(10):
        step(each, capacity)
    end.record()
    torch.cuda.synchronize()
    rr.check_kernel_error()
    print(f"{begin.elapsed_time(end) / 10 * 1000:.0f} us a step of {a.ranks} ranks")
    return far


if __name__ == "__main__":
    main()
