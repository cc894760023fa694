"""Training steps and single-token decoding of a small language model with an expert layer,
every matrix product of it a call of this library:

    python examples/expert_lm_step.py [steps]

Token embedding -> feed-forward block (linear + GELU, linear + residual) -> expert layer (top-1
router, rows sorted by expert, grouped products, residual) -> cross entropy of the output
head, without logits.  Weights are FP32 masters with BF16 copies for the products; the
optimizer is plain SGD.  The synthetic task: the next token is a fixed permutation of the
current one.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_tensor_gb300 as tcg  # noqa: E402

BF16 = torch.bfloat16


class Model:
    def __init__(self, vocab=1003, hidden=128, wide=256, experts=6, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape, fan):
            return torch.randn(*shape, generator=g, device=device) / fan ** 0.5

        self.experts = experts
        self.params = {
            "embed": weight(vocab, hidden, fan=1.0),
            "w1": weight(wide, hidden, fan=hidden), "b1": torch.zeros(wide, device=device),
            "w2": weight(hidden, wide, fan=wide), "b2": torch.zeros(hidden, device=device),
            "router": weight(experts, hidden, fan=hidden),
            "e1": weight(experts, wide, hidden, fan=hidden),
            "c1": torch.zeros(experts, wide, device=device),
            "e2": weight(experts, hidden, wide, fan=wide),
            "head": weight(vocab, hidden, fan=hidden),
        }
        self.handle = tcg.Handle()
        self.refresh()

    def refresh(self):
        """The BF16 copies that the products read."""
        self.w = {k: v.to(BF16) for k, v in self.params.items()}

    def forward(self, tokens):
        """Hidden states before the head, and what the backward pass needs."""
        h, w = self.handle, self.w
        s = {"tokens": tokens, "x0": w["embed"][tokens]}
        rows = tokens.shape[0]
        # feed-forward block with the residual in the second product's epilogue
        s["z1"] = s["x0"].new_empty(rows, w["w1"].shape[0])
        s["a1"] = tcg.linear(h, s["x0"], w["w1"], bias=w["b1"], act="gelu", z=s["z1"])
        s["x1"] = tcg.linear(h, s["a1"], w["w2"], bias=w["b2"], residual=s["x0"])
        # router: each row to the expert with the largest probability; rows sorted by expert
        s["p"] = torch.softmax(tcg.linear(h, s["x1"], w["router"], out_dtype=torch.float32), 1)
        s["gate"], s["choice"] = s["p"].max(1)
        s["order"] = torch.argsort(s["choice"], stable=True)
        counts = torch.bincount(s["choice"], minlength=self.experts)
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
        s["xs"] = s["x1"][s["order"]]
        s["ze"] = s["xs"].new_empty(rows, w["e1"].shape[1])
        s["ae"] = tcg.grouped_linear(h, s["xs"], w["e1"], s["offsets"], bias=w["c1"], act="silu",
                                     z=s["ze"])
        s["ys"] = tcg.grouped_linear(h, s["ae"], w["e2"], s["offsets"])
        y = torch.empty_like(s["ys"])
        y[s["order"]] = (s["ys"].float() * s["gate"][s["order"], None]).to(BF16)
        s["x2"] = s["x1"] + y
        return s

    def backward(self, s, dx2):
        """Gradients of all parameters but the head's, given that of the hidden states."""
        h, w, g = self.handle, self.w, {}
        order, gate = s["order"], s["gate"]
        dys = dx2[order]
        dgate = torch.empty_like(gate)
        dgate[order] = (dys.float() * s["ys"].float()).sum(1)
        dys = (dys.float() * gate[order, None]).to(BF16)
        dae, g["e2"], _ = tcg.grouped_linear_backward(h, dys, s["ae"], w["e2"], s["offsets"],
                                                      want=("dx", "dw"))
        dxs, g["e1"], g["c1"] = tcg.grouped_linear_backward(h, dae, s["xs"], w["e1"], s["offsets"],
                                                            z=s["ze"], act="silu")
        dx1 = dx2.clone()
        dx1[order] += dxs
        # d softmax of the chosen probability
        dlogits = -s["p"] * (gate * dgate)[:, None]
        dlogits.scatter_add_(1, s["choice"][:, None], (gate * dgate)[:, None])
        rows = dx1.shape[0]
        padded = dlogits.new_zeros(rows, (self.experts + 7) // 8 * 8, dtype=BF16)
        padded[:, :self.experts] = dlogits
        dxr, g["router"], _ = tcg.linear_backward(h, padded[:, :self.experts], s["x1"], w["router"],
                                                  want=("dx", "dw"))
        dx1 += dxr
        da1, g["w2"], g["b2"] = tcg.linear_backward(h, dx1, s["a1"], w["w2"])
        dx0, g["w1"], g["b1"] = tcg.linear_backward(h, da1, s["x0"], w["w1"], z=s["z1"], act="gelu")
        dx0 += dx1
        g["embed"] = torch.zeros_like(self.params["embed"]).index_add_(0, s["tokens"], dx0.float())
        return g

    def loss_and_gradients(self, tokens, targets):
        s = self.forward(tokens)
        loss, lse = tcg.linear_cross_entropy(self.handle, s["x2"], self.w["head"], targets)
        count = (targets >= 0).sum()
        dloss = (1.0 / count).expand(tokens.shape[0]).contiguous()
        dx2, dhead = tcg.linear_cross_entropy_backward(self.handle, s["x2"], self.w["head"], targets,
                                                       lse, dloss)
        grads = self.backward(s, dx2)
        grads["head"] = dhead
        return loss.sum() / count, grads

    def step(self, tokens, targets, rate):
        loss, grads = self.loss_and_gradients(tokens, targets)
        for name, p in self.params.items():
            p -= rate * grads[name].float()
        self.refresh()
        return loss

    def decode(self, token, steps):
        """Greedy decoding, one token at a time."""
        out = []
        for _ in range(steps):
            s = self.forward(token)
            logits = tcg.linear(self.handle, s["x2"], self.w["head"], out_dtype=torch.float32)
            token = logits.argmax(1)
            out.append(token)
        return torch.cat(out)


def train(steps=60, rows=2048, rate=4.0, seed=0, vocab=1003):
    """(losses, share of tokens that decoding gets right)."""
    model = Model(vocab=vocab, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    following = torch.randperm(vocab, generator=g, device="cuda")
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        targets = following[tokens]
        targets[::50] = -100                           # padding takes no part
        losses.append(model.step(tokens, targets, rate))
    start = torch.randint(0, vocab, (1,), generator=g, device="cuda")
    said = model.decode(start, 20)
    truth = torch.cat([start, said[:-1]])
    tcg.check(tcg.tcg_get_device_error(model.handle.h), "device error word")
    return torch.stack(losses).tolist(), float((following[truth] == said).float().mean())


if __name__ == "__main__":
    losses, right = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i in range(0, len(losses), 10):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"last loss {losses[-1]:.4f}, decoded tokens right: {100 * right:.0f}%")
