"""The MXFP4 operators together, as a decoding program uses them.

A residual stack of MoE layers and a vocabulary projection, all weights
quantized to MXFP4 once; a prompt runs through it with 4-bit activations
(quantize, grouped products, the vocabulary's product), then tokens are drawn
one at a time with 16-bit activations (the few-token layer and the few-row
product).  Between the layers the residual stream takes the last one's output
and is normed for the next, the last time into MXFP4 for the vocabulary.  The weights
are random: the point is the calls, not the text.

  python examples/mx4_generate.py [--layers 4] [--prompt 300] [--steps 32]
                                  [--scores] [--adapter]

--scores routes by sigmoid scores with groups of experts, --adapter adds a
low-rank adapter to the vocabulary's projection."""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_sparse_moe_gb300 as qsm  # noqa: E402

H, I, E, K, VOCAB = 2048, 512, 64, 8, 32000


def random_layer(gen):
    def w(*shape):
        return (torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(torch.bfloat16)
    return qsm.Mx4Layer.quantize(H, I, E, K, w(E, 2 * I, H), w(E, H, I), w(1, 2 * I, H), w(1, H, I),
                                 torch.randn((E, H), generator=gen, device="cuda") * 0.05)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--scores", action="store_true")
    ap.add_argument("--adapter", action="store_true")
    a = ap.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    layers = [random_layer(gen) for _ in range(a.layers)]
    embed = torch.randn((VOCAB, H), generator=gen, device="cuda").to(torch.bfloat16)
    head = qsm.mx4_quantize(embed)                      # the projection shares the embedding
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    norm = qsm.ResidualNorm(H, pre=qsm.Norm())          # x + y, and its norm
    routers = [qsm.MoERouter(layer.w_router, K, "sigmoid", groups=8, groups_kept=4, group_best=2) if a.scores else None
               for layer in layers]
    adapters = None
    if a.adapter:
        adapters = qsm.LoraAdapters((torch.randn((1, 16, H), generator=gen, device="cuda") * H ** -0.5).to(torch.bfloat16),
                                    (torch.randn((1, VOCAB, 16), generator=gen, device="cuda") * 0.25).to(torch.bfloat16))

    def stack(x, forward, last):
        """The layers on x, and the normed result (a dtype, or "mx4")."""
        _, h = norm(x)
        for n, f in enumerate(forward):
            x, h = norm(x, f(h), x_out=x, h=last if n + 1 == len(forward) else None, dev_status=status)
        return h

    def adapted(logits, h):
        if adapters is None:
            return logits
        ids = torch.zeros(len(logits), dtype=torch.int32, device="cuda")
        return qsm.lora_add(h, adapters, ids, logits, out=logits, dev_status=status)

    # the prompt: every layer on all its tokens, 4-bit activations
    prompt = torch.randint(0, VOCAB, (a.prompt,), generator=gen, device="cuda")
    forward = [qsm.Mx4Forward(layer, a.prompt, acts="mx4", router=r) for layer, r in zip(layers, routers)]
    h = stack(embed[prompt], forward, "mx4")
    logits = qsm.mx4_gemm(h, head, dev_status=status)
    token = adapted(logits, qsm.mx4_dequantize(h))[-1:].argmax(dim=1)

    # one token at a time, 16-bit activations
    decode = [qsm.Mx4Forward(layer, 1, acts="bf16", router=r) for layer, r in zip(layers, routers)]
    tokens = [token]
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        h = stack(embed[token], decode, torch.bfloat16)
        token = adapted(qsm.mx4_gemv(h, head, dev_status=status), h).argmax(dim=1)
        tokens.append(token)
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    bits = status.item()
    for f in forward + decode:
        bits |= f.dev_status.item()
    if bits:
        raise SystemExit(f"device status {bits}")
    print(f"prompt of {a.prompt} tokens, {a.steps} tokens drawn at {a.steps / took:.0f} a second, "
          f"first {torch.cat(tokens)[:8].tolist()}")


if __name__ == "__main__":
    main()
