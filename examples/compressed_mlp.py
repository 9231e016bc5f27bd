"""A gated MLP compressed two ways and run token by token.

The MLP is y = (act(x Wg^T) * (x Wu^T)) Wd^T.  Calibration tokens go through
the dense gated block; the second moments of its output are the importance that
the ternary decomposition of Wd takes.  Gate and up projection become 4-bit
weights, tuned first by a few AdamW steps through the gated block so that
their quantized form reproduces the dense outputs.  The output projection is
tuned behind them, a linear layer on the compressed block's h, so that what is
compressed of it makes up for what the 4 bits lost.  Then single tokens run
through the compressed layer: q4_gated for gate and up, q4_apply or the ternary
factors' apply_rows for down.

    python examples/compressed_mlp.py [--hidden 2432] [--width 640] [--tokens 512]

Needs an MI355X; weights and tokens are synthetic.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import synthetic  # noqa: E402
import ternary_rank_weight_amd as trw  # noqa: E402


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def quantized(w, group):
    """The bf16 values that w's 4-bit form stands for, and that form."""
    q = trw.q4_quantize(w, group, symmetric=False)
    return trw.q4_reconstruct(q, torch.bfloat16), q


def tune(x, target, wg, wu, group, steps, rate):
    """Gate and up weights whose 4-bit values bring h(x) nearer to target: gradients are taken at
    the quantized values and applied to the weights behind them."""
    wg, wu = (w.float().clone() for w in (wg, wu))
    # steps measured in the weights' own size
    opts = [trw.AdamW([w], lr=float(rate * w.abs().mean()), betas=(0.8, 0.95), weight_decay=0.0) for w in (wg, wu)]
    for _ in range(steps):
        leaves = [quantized(w, group)[0].requires_grad_() for w in (wg, wu)]
        h = trw.gated(x, *leaves)
        loss = (h.float() - target.float()).square().mean() / target.float().square().mean()
        for opt, grad in zip(opts, torch.autograd.grad(loss, leaves)):
            opt.step([grad])
    return wg, wu


def output_loss(h, wd, target):
    y = trw.linear(h, wd)
    return (y.float() - target.float()).square().mean() / target.float().square().mean()


def tune_output(h, target, wd, steps, rate):
    """The output projection whose y = h Wd^T is nearer to target: bf16 weights with fp32 masters and
    moments of 8 bits."""
    wd = wd.clone().requires_grad_()
    opt = trw.AdamW([wd], lr=float(rate * wd.detach().float().abs().mean()), betas=(0.8, 0.95), weight_decay=0.0,
                    bits=8, master=True)
    for _ in range(steps):
        opt.step(torch.autograd.grad(output_loss(h, wd, target), [wd]))
    return wd.detach()


def run(hidden=2432, width=640, tokens=512, group=32, steps=10, mu=2.0, seed=0):
    device = "cuda"
    wg, wu, wd = (torch.from_numpy(synthetic.llm_like(m, n, seed + i)).to(device)
                  for i, (m, n) in enumerate([(hidden, width), (hidden, width), (width, hidden)]))
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    x = torch.randn(tokens, width, generator=gen, device=device).bfloat16()
    g16, u16, d16 = wg.bfloat16(), wu.bfloat16(), wd.bfloat16()
    h = trw.gated_forward(x, g16, u16)

    # gate and up in 4 bits, before and after tuning
    plain = trw.q4_gated(quantized(wg, group)[1], quantized(wu, group)[1], x)
    tg, tu = tune(x, h, wg, wu, group, steps, rate=0.005)
    qg, qu = quantized(tg, group)[1], quantized(tu, group)[1]
    tuned = trw.q4_gated(qg, qu, x)

    # down, behind the compressed gate and up
    hq = trw.gated_forward(x, trw.q4_reconstruct(qg, torch.bfloat16), trw.q4_reconstruct(qu, torch.bfloat16))
    y = trw.linear_forward(h, d16)
    t16 = tune_output(hq, y, d16, steps, rate=0.005)
    behind = relative(trw.linear_forward(hq, d16), y), relative(trw.linear_forward(hq, t16), y)

    # down: 4 bits, and ternary factors weighted by the calibration's second moments
    qd = trw.q4_quantize(wd, group, symmetric=False)
    importance = h.float().square().mean(0)
    res = trw.decompose(wd, mu, 0.7, block=64, importance=importance, lam=0.05)
    bt2 = trw.transpose_codes(res.B2, res.k, width)

    # one token through each layer
    one = x[:1]
    dense = trw.linear_forward(trw.gated_forward(one, g16, u16), d16)
    h1 = trw.q4_gated(qg, qu, one)
    four_bit = trw.q4_apply(qd, h1)
    ternary = trw.apply_rows(bt2, res.C2, res.D, width, hidden, h1.float().view(-1))
    err = 1 - relative(trw.q4_reconstruct(qd), wd) ** 2
    return {"h_4bit": relative(plain, h), "h_4bit_tuned": relative(tuned, h),
            "y_h_4bit": behind[0], "y_h_4bit_tuned": behind[1],
            "y_4bit": relative(four_bit, dense), "y_ternary": relative(ternary.view(1, -1), dense),
            "energy_4bit": err, "energy_ternary": float(res.energy.item())}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=2432)
    ap.add_argument("--width", type=int, default=640)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    r = run(a.hidden, a.width, a.tokens, steps=a.steps)
    print(f"h = act(g) u of {a.tokens} tokens, 4-bit gate and up: error {r['h_4bit']:.4f}, tuned {r['h_4bit_tuned']:.4f}")
    print(f"y behind them, dense down: error {r['y_h_4bit']:.4f}, tuned {r['y_h_4bit_tuned']:.4f}")
    print(f"down projection: 4-bit energy {r['energy_4bit']:.5f}, ternary weighted energy {r['energy_ternary']:.5f}")
    print(f"one token's y: 4-bit layer error {r['y_4bit']:.4f}, ternary down {r['y_ternary']:.4f}")


if __name__ == "__main__":
    main()
