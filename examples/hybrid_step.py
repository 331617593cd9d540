"""A hybrid model's verify steps: recurrent layers and attention layers over one prompt and its drafts.

    python examples/hybrid_step.py [--prompt 1000] [--steps 4] [--cache e4m3] [--rope] [--gates] [--temperature 0.7 [--top-k 40] [--top-p 0.9]]

Every step verifies a block of T draft tokens. Each recurrent layer keeps a state checkpoint per position;
each attention layer appends the block's keys and values to its paged cache and attends over it. One greedy
accept decides for all of them: the recurrent layers commit the checkpoint of the accepted position, and the
attention layers' cache is rolled back by shortening kv_len. Both read the accepted length on the device, so
nothing waits for the host. The residual stream between the layers is added to and normed in one call. With --rope the
attention layers turn queries and keys by their positions on the way to the cache, with --gates every head's output is gated (and, in a recurrent
layer, normed), and with --temperature the accept draws its targets instead of taking the largest. The projections between
are random matrices: there is no checkpoint to load.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from deltanet_recurrent_state_gb300 import binding as dn  # noqa: E402

HIDDEN, VOCAB, T = 1024, 4096, 16
HEADS, DIM = 8, 128                       # recurrent layers: state DIM x DIM a head
Q_HEADS, KV_HEADS, HEAD_DIM, PAGE = 16, 4, 128, 64  # attention layers
ROTATED, EPS = 64, torch.finfo(torch.float16).eps


class HybridModel:
    """Alternating recurrent and attention layers with random weights, fp16, one request."""

    def __init__(self, layers=4, max_tokens=4096, cache="f16", seed=0, device="cuda", rope=False, gates=False):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.device = device

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * rows ** -0.5).half()

        self.embed, self.head = torch.randn((VOCAB, HIDDEN), generator=g, device=device).half(), weight(HIDDEN, VOCAB)
        self.last = torch.zeros(1, dtype=torch.int64, device=device)  # the newest token, not yet run
        self.layers = []
        pages = -(-max_tokens // PAGE)
        for i in range(layers):
            if i % 2 == 0:
                d = dict(kind="recurrent", qkv=weight(HIDDEN, 3 * HEADS * DIM), gates=weight(HIDDEN, 2 * HEADS), out=weight(HEADS * DIM, HIDDEN),
                         state=torch.zeros((1, HEADS, DIM, DIM), dtype=torch.float16, device=device), width=(HEADS, DIM))
            else:
                d = dict(kind="attention", qkv=weight(HIDDEN, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM), out=weight(Q_HEADS * HEAD_DIM, HIDDEN),
                         width=(Q_HEADS, HEAD_DIM))
                shape = (pages, KV_HEADS, PAGE, HEAD_DIM)
                for x in "kv":
                    if cache == "e4m3":
                        d[x] = torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                        d[x + "_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device=device)
                    else:
                        d[x], d[x + "_exp"] = torch.zeros(shape, dtype=torch.float16, device=device), None
            if gates:
                d["gate"] = weight(HIDDEN, d["width"][0] * d["width"][1])
            self.layers.append(d)
        self.freqs = dn.rope_freqs(ROTATED, device=device)[0] if rope else None
        # one page table for all attention layers: their pools are laid out alike
        self.page_table = torch.randperm(pages, generator=g, device=device).to(torch.int32)[None, :].contiguous()
        self.kv_len = torch.zeros(1, dtype=torch.int32, device=device)

    def forward(self, tokens, commit_all):
        """Logits [n, VOCAB] of n new tokens; commit_all: a prompt's tokens (else a verify block of T)."""
        n = tokens.numel()
        self.kv_len += n
        start = torch.tensor([0, n], dtype=torch.int32, device=self.device)
        x = self.embed[tokens]
        h, _ = dn.dn_residual_norm(None, x, eps=EPS)
        for i, d in enumerate(self.layers):
            if d["kind"] == "recurrent":
                q, k, v = (h @ d["qkv"]).view(1, n, 3 * HEADS, DIM).split(HEADS, dim=2)
                q, k = (torch.nn.functional.normalize(z.float(), dim=-1).half() for z in (q, k))
                beta, decay = (h @ d["gates"]).float().view(1, n, 2, HEADS).unbind(2)
                beta, decay = torch.sigmoid(beta).contiguous(), torch.sigmoid(decay + 3).contiguous()
                if commit_all:
                    o, _, _ = dn.dn_prefill_checkpoint(q, k, v.contiguous(), beta, decay, state_in=d["state"], state_out=d["state"])
                else:
                    o, d["ckpt"] = dn.dn_verify_block(q, k, v.contiguous(), beta, decay, d["state"])
                o, order, act = o[0], "norm_gate", "silu"
            else:
                # the three are slices of one projection: the calls take row strides
                q, k, v = (h @ d["qkv"]).view(n, -1, HEAD_DIM).split((Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
                where = (start, self.kv_len, self.page_table, d["k"], d["v"], d["k_exp"], d["v_exp"])
                if self.freqs is None:
                    dn.dn_kv_append(k, v, *where)
                else:
                    q = dn.dn_rope_append(q, k, v, self.freqs, *where)
                o, _ = dn.dn_attn_paged(q, *where)
                order, act = "gate", "sigmoid"
            if "gate" in d:
                o = dn.dn_head_norm(o, (h @ d["gate"]).view(o.shape), order=order, act=act)
            y = o.reshape(n, -1) @ d["out"]
            if i + 1 < len(self.layers):
                h, _ = dn.dn_residual_norm(y, x, eps=EPS)  # x is added to in place, and the next layer reads its norm
            else:
                x += y  # (this model's head reads the stream itself)
        return x @ self.head

    def prompt(self, tokens):
        """Run all but the last token of a prompt; the last one begins the first verify block."""
        if tokens.numel() > 1:
            self.forward(tokens[:-1], commit_all=True)
        self.last = tokens[-1:]

    def verify(self, drafts, uniform=None, **filters):
        """One verify step of T drafts: (the model's own tokens [T], accepted length [1]), both on the device.

        With random numbers uniform [T] the model's tokens are drawn, with the filters (temperature, top_k, ..) of dn_accept_sampled.

        The block runs the newest token and all drafts but the last, so position t says what the model
        would have in the place of draft t.
        """
        logits = self.forward(torch.cat([self.last, drafts[:-1].long()]), commit_all=False)
        logits, drafts_1 = logits.view(1, T, VOCAB), drafts.view(1, T)
        if uniform is None:
            target, accepted = dn.dn_accept_greedy(logits, drafts_1)
        else:
            target, accepted, _ = dn.dn_accept_sampled(logits, drafts_1, uniform.view(1, T), **filters)
        for d in self.layers:
            if d["kind"] == "recurrent":
                dn.dn_commit(d.pop("ckpt"), accepted, d["state"])
        self.kv_len += accepted - T  # what was rejected is no longer cached
        newest = drafts.long().gather(0, (accepted.long() - 1).clamp(min=0))
        self.last = torch.where(accepted > 0, newest, self.last)
        return target[0], accepted


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--cache", choices=["f16", "e4m3"], default="f16")
    ap.add_argument("--rope", action="store_true", help="turn queries and keys by their positions")
    ap.add_argument("--gates", action="store_true", help="gate every head's output")
    ap.add_argument("--temperature", type=float, default=0.0, help="draw the model's tokens (0: take the largest)")
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=1.0)
    args = ap.parse_args()
    if args.prompt < 1:
        ap.error("a prompt has a token at least")
    model = HybridModel(cache=args.cache, max_tokens=args.prompt + T * (args.steps + 1), rope=args.rope, gates=args.gates)
    filters = dict(temperature=torch.tensor([args.temperature], device="cuda"), top_k=torch.tensor([args.top_k], dtype=torch.int32, device="cuda"),
                   top_p=torch.tensor([args.top_p], device="cuda"))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    model.prompt(torch.randint(0, VOCAB, (args.prompt,), generator=g, device="cuda"))
    drafts = torch.randint(0, VOCAB, (T,), generator=g, device="cuda", dtype=torch.int32)
    for step in range(args.steps):
        uniform = torch.rand(T, generator=g, device="cuda") if args.temperature > 0 else None
        target, accepted = model.verify(drafts, uniform, **filters) if uniform is not None else model.verify(drafts)
        print("step %d: accepted %d of %d drafts, %d tokens cached; the model's own token is %d"
              % (step, int(accepted), T, int(model.kv_len), int(target[min(int(accepted), T - 1)])))
        # the next drafts: what the model itself had from the first rejected place on, then its last word again
        drafts = target[(torch.arange(T, device="cuda") + accepted).clamp(max=T - 1)].contiguous()


if __name__ == "__main__":
    main()
