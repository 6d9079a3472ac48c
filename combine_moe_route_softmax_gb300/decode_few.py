"""A decode step of a few tokens, as a serving program would run it: a stack of MoE layers
(moe_layer_few, the router inside or ahead of it), then an output head in 4 bits
(moe_linear_w4) and the largest logit of each token.

    python -m combine_moe_route_softmax_gb300.decode_few --tokens 4 --layers 4 --weights w4

Weights and tokens are random: the next hidden state is a row of a random table, so the numbers
printed are times and the agreement of the two ways of routing, not text.
"""
import argparse

import torch

import combine_moe_route_softmax_gb300 as moe

FORMATS = {"bf16": moe.MOE_BF16, "e4m3": moe.MOE_E4M3, "w4": moe.MOE_W4}


class DecodeStep:
    """Weights, workspaces and buffers of the step for up to `tokens` tokens, made once."""

    def __init__(self, tokens, layers, H, I, E, K, vocab, weights="w4", group=128, shared=True, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(*shape):
            w = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
            for m in w.view(-1, *shape[-2:]):          # one at a time: no float32 copy of the stack
                m.copy_(torch.randn(m.shape, generator=g, device="cuda") * shape[-1] ** -0.5)
            return w

        self.K = K
        self.routers = [matrix(E, H) for _ in range(layers)]
        self.inside, self.outside = [], []             # the same layers with and without a router
        for wr in self.routers:
            kw = {}
            names = ["w13", "w2"] + (["shared_w13", "shared_w2"] if shared else [])
            for name in names:
                lead = () if name.startswith("shared") else (E,)
                w = matrix(*lead, *((2 * I, H) if name.endswith("w13") else (H, I)))
                if weights == "w4":
                    kw[name] = moe.moe_pack_w4(*moe.moe_quantize_weight_w4(w, group))
                elif weights == "e4m3":
                    kw[name], kw[name + "_scales"] = moe.moe_quantize_weight_fp8(w)
                else:
                    kw[name] = w
            self.inside.append(moe.MoeLayerFew(tokens, H, I, E, K, FORMATS[weights], w_router=wr, **kw))
            self.outside.append(moe.MoeLayerFew(tokens, H, I, E, K, FORMATS[weights], **kw))
        self.head = moe.moe_pack_w4(*moe.moe_quantize_weight_w4(matrix(vocab, H), group, zeros=True))
        self.head_ws = moe.moe_linear_w4_workspace(tokens, vocab, H)
        self.route_ws = moe.moe_route_hidden_workspace()
        self.table = matrix(vocab, H) * H ** 0.5       # next token -> its hidden state
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def __call__(self, x, route_inside=True):
        """x BF16 [t, H] -> (logits float32 [t, vocab], the layers' expert ids)."""
        ids = []
        for wr, inside, outside in zip(self.routers, self.inside, self.outside):
            if route_inside:
                y, idx, _ = inside.forward(x, dev_status=self.status)
            else:
                # where the ids are wanted before the experts run (to count or fetch them)
                idx, w, _ = moe.moe_route_hidden(x, wr, self.K, ws=self.route_ws)
                y, _, _ = outside.forward(x, topk_idx=idx, topk_w=w, dev_status=self.status)
            x = x + y
            ids.append(idx)
        return moe.moe_linear_w4(x, self.head, out_dtype=torch.float32, ws=self.head_ws, dev_status=self.status), ids

    def capture(self, x, route_inside=True):
        """A CUDA graph that decodes one token per row: x becomes the next hidden states in place."""
        self(x, route_inside)                          # nothing is set up for the first time while capturing
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            logits, _ = self(x, route_inside)
            x.copy_(self.table[logits.argmax(1)])
        return graph


def run(tokens=4, layers=2, H=2048, I=1408, E=64, K=8, vocab=32768, weights="w4", group=128, steps=20, seed=0):
    """Decodes `steps` tokens per row both ways; returns the milliseconds per step and whether
    both gave the same bits."""
    step = DecodeStep(tokens, layers, H, I, E, K, vocab, weights, group, seed=seed)
    start = step.table[:tokens].clone()
    ms, ends = {}, []
    for inside in (True, False):
        x = start.clone()
        graph = step.capture(x, inside)
        x.copy_(start)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for _ in range(3):
            graph.replay()
        x.copy_(start)
        begin.record()
        for _ in range(steps):
            graph.replay()
        end.record()
        end.synchronize()
        ms["router in the layer" if inside else "router ahead"] = begin.elapsed_time(end) / steps
        ends.append(x)
    if step.status.item():
        raise RuntimeError(f"device status {step.status.item()}")
    return ms, torch.equal(*ends)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 4), ("layers", 4), ("hidden", 2048), ("intermediate", 1408), ("experts", 64),
                        ("topk", 8), ("vocab", 32768), ("group", 128), ("steps", 50)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--weights", choices=sorted(FORMATS), default="w4")
    a = p.parse_args(argv)
    ms, same = run(a.tokens, a.layers, a.hidden, a.intermediate, a.experts, a.topk, a.vocab, a.weights, a.group, a.steps)
    for name, t in ms.items():
        print(f"{a.weights}, {a.tokens} tokens, {a.layers} layers, {name}: {t:.3f} ms per step, "
              f"{a.tokens / t * 1e3:.0f} tokens/s")
    print("both ways give the same bits" if same else "THE TWO WAYS DIFFER")
    return 0 if same else 1


if __name__ == "__main__":
    raise SystemExit(main())
