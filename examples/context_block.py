"""A residual block in which nodes attend to a context, and its training step.

    y = x + dropout(W_o attention(W_q norm(x), W_k c, W_v c))

x holds the node rows of a batch of systems laid end to end, c the rows of each
system's context (any number of them, none included). The maps are equivariant
linear maps, so y turns with x and c. The backward pass is written out, each
layer's own in reverse order.

    python -m examples.context_block
"""

import torch

from clebsch_gordan_tensor_amd import cgtp, layers


def head_irreps(irreps, heads, kv_heads):
    """The context's irreps: kv_heads / heads of every multiplicity."""
    blocks = [block.strip().split("x") for block in irreps.split("+")]
    return "+".join("%dx%s" % (int(mul) // heads * kv_heads, kind) for mul, kind in blocks)


def random_weights(lin, gen):
    """Normal weights of variance 1 / inputs, path by path."""
    parts = [torch.randn(u * v, generator=gen, device="cuda") * u ** -0.5 for _, _, _, u, v in lin.paths().tolist()]
    return torch.cat(parts).to(lin.torch_dtype)


class Layout:
    """The sample layouts of a batch: offsets of each system's node and context rows."""

    def __init__(self, block, node_ptr, context_ptr):
        self.nodes, self.context = layers.Samples(node_ptr), layers.Samples(context_ptr)
        self.batch = block.attn.batch(self.nodes, self.context)


class ContextBlock:
    """Weights are tensors in ``params``; gradients come back under the same names."""

    def __init__(self, irreps, context_irreps, heads, kv_heads, groups, p=0.1, dtype="f32", seed=0):
        kv = head_irreps(irreps, heads, kv_heads)
        self.p, self.seed = p, seed
        self.norm = layers.GroupNorm(irreps, groups, activation="silu", dtype=dtype)
        self.to_q = cgtp.Linear(irreps, irreps, dtype=dtype)
        self.to_kv = cgtp.Linear(context_irreps, kv + "+" + kv, dtype=dtype)    # a row holds k, then v
        self.attn = layers.CrossAttention(irreps, heads, kv_heads, dtype=dtype)
        self.to_out = cgtp.Linear(irreps, irreps, dtype=dtype)
        self.drop = layers.Dropout(irreps, dtype=dtype)
        dt, gen = self.norm.torch_dtype, torch.Generator(device="cuda").manual_seed(seed)
        self.params = {
            "norm_w": torch.ones(self.norm.channels, device="cuda", dtype=dt),
            "norm_b": torch.zeros(self.norm.biases, device="cuda", dtype=dt),
            "w_q": random_weights(self.to_q, gen),
            "w_kv": random_weights(self.to_kv, gen),
            "w_out": random_weights(self.to_out, gen),
        }

    def forward(self, layout, x, c, step, key_mask=None):
        """(y, what the backward takes); ``step`` differs from call to call (the dropout's offset)."""
        w, dk = self.params, self.attn.dim_kv
        n, stats = self.norm.forward(layout.nodes, x, w["norm_w"], w["norm_b"])
        q = self.to_q.forward(n, w["w_q"])
        kv = self.to_kv.forward(c, w["w_kv"])
        a, lse = self.attn.forward(layout.batch, q, kv[:, :dk], kv[:, dk:], key_mask=key_mask, need_lse=True)
        y = self.drop.forward(self.to_out.forward(a, w["w_out"]), self.p, self.seed, step, residual=x)
        return y, (layout, x, c, step, key_mask, n, stats, q, kv, a, lse)

    def backward(self, saved, grad_y):
        """(grad_x, grad_c, the parameters' gradients)."""
        layout, x, c, step, key_mask, n, stats, q, kv, a, lse = saved
        w, dk, g = self.params, self.attn.dim_kv, {}
        gu = self.drop.backward(grad_y, self.p, self.seed, step)
        ga, g["w_out"] = self.to_out.backward(a, w["w_out"], gu)
        gq, gk, gv = self.attn.backward(layout.batch, q, kv[:, :dk], kv[:, dk:], a, lse, ga, key_mask=key_mask)
        gc, g["w_kv"] = self.to_kv.backward(c, w["w_kv"], torch.cat([gk, gv], 1))
        gn, g["w_q"] = self.to_q.backward(n, w["w_q"], gq)
        gx, g["norm_w"], g["norm_b"] = self.norm.backward(layout.nodes, x, w["norm_w"], w["norm_b"], stats, gn)
        return gx + grad_y, gc, g


def main(steps=40, rate=0.3):
    """Fit a block to the outputs of another one on ragged systems; prints the loss."""
    irreps, context = "32x0e+32x1o+32x2e", "16x0e+16x1o+16x2e"
    teacher, block = (ContextBlock(irreps, context, 4, 2, 4, p=p, seed=s) for p, s in ((0.0, 1), (0.05, 2)))
    node_ptr, context_ptr = [0, 21, 30, 51], [0, 40, 40, 73]                  # the second system has no context
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((node_ptr[-1], block.norm.dim), generator=gen, device="cuda")
    c = torch.randn((context_ptr[-1], block.to_kv.dim_in), generator=gen, device="cuda")
    target = teacher.forward(Layout(teacher, node_ptr, context_ptr), x, c, 0)[0]
    layout, losses = Layout(block, node_ptr, context_ptr), []
    for step in range(steps):
        y, saved = block.forward(layout, x, c, step)
        diff = y - target
        losses.append(float((diff * diff).mean()))
        grads = block.backward(saved, diff * (2.0 / x.shape[0]))[2]
        for name, p in block.params.items():
            p -= rate * grads[name] / block.norm.dim ** 0.5
        if step % 10 == 0 or step == steps - 1:
            print("step %3d  loss %.5f" % (step, losses[-1]), flush=True)
    return losses


if __name__ == "__main__":
    main()
