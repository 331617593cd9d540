"""A hybrid model's verify steps: recurrent layers and attention layers over one prompt and its drafts.

    python examples/hybrid_step.py [--prompt 1000] [--steps 4] [--cache e4m3]

Every step verifies a block of T draft tokens. Each recurrent layer keeps a state checkpoint per position;
each attention layer appends the block's keys and values to its paged cache and attends over it. One greedy
accept decides for all of them: the recurrent layers commit the checkpoint of the accepted position, and the
attention layers' cache is rolled back by shortening kv_len. Both read the accepted length on the device, so
nothing waits for the host. The projections between are random matrices: there is no checkpoint to load.
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


class HybridModel:
    """Alternating recurrent and attention layers with random weights, fp16, one request."""

    def __init__(self, layers=4, max_tokens=4096, cache="f16", seed=0, device="cuda"):
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
                         state=torch.zeros((1, HEADS, DIM, DIM), dtype=torch.float16, device=device))
            else:
                d = dict(kind="attention", qkv=weight(HIDDEN, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM), out=weight(Q_HEADS * HEAD_DIM, HIDDEN))
                shape = (pages, KV_HEADS, PAGE, HEAD_DIM)
                for x in "kv":
                    if cache == "e4m3":
                        d[x] = torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                        d[x + "_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device=device)
                    else:
                        d[x], d[x + "_exp"] = torch.zeros(shape, dtype=torch.float16, device=device), None
            self.layers.append(d)
        # one page table for all attention layers: their pools are laid out alike
        self.page_table = torch.randperm(pages, generator=g, device=device).to(torch.int32)[None, :].contiguous()
        self.kv_len = torch.zeros(1, dtype=torch.int32, device=device)

    def forward(self, tokens, commit_all):
        """Logits [n, VOCAB] of n new tokens; commit_all: a prompt's tokens (else a verify block of T)."""
        n = tokens.numel()
        self.kv_len += n
        start = torch.tensor([0, n], dtype=torch.int32, device=self.device)
        x = self.embed[tokens]
        for d in self.layers:
            y = torch.nn.functional.rms_norm(x, (HIDDEN,))
            if d["kind"] == "recurrent":
                q, k, v = (y @ d["qkv"]).view(1, n, 3 * HEADS, DIM).split(HEADS, dim=2)
                q, k = (torch.nn.functional.normalize(z.float(), dim=-1).half() for z in (q, k))
                beta, decay = (y @ d["gates"]).float().view(1, n, 2, HEADS).unbind(2)
                beta, decay = torch.sigmoid(beta).contiguous(), torch.sigmoid(decay + 3).contiguous()
                if commit_all:
                    o, _, _ = dn.dn_prefill_checkpoint(q, k, v.contiguous(), beta, decay, state_in=d["state"], state_out=d["state"])
                else:
                    o, d["ckpt"] = dn.dn_verify_block(q, k, v.contiguous(), beta, decay, d["state"])
                y = o.view(n, HEADS * DIM)
            else:
                # the three are slices of one projection: the calls take row strides
                q, k, v = (y @ d["qkv"]).view(n, -1, HEAD_DIM).split((Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
                where = (start, self.kv_len, self.page_table, d["k"], d["v"], d["k_exp"], d["v_exp"])
                dn.dn_kv_append(k, v, *where)
                o, _ = dn.dn_attn_paged(q, *where)
                y = o.view(n, Q_HEADS * HEAD_DIM)
            x = x + y @ d["out"]
        return x @ self.head

    def prompt(self, tokens):
        """Run all but the last token of a prompt; the last one begins the first verify block."""
        if tokens.numel() > 1:
            self.forward(tokens[:-1], commit_all=True)
        self.last = tokens[-1:]

    def verify(self, drafts):
        """One verify step of T drafts: (the model's own tokens [T], accepted length [1]), both on the device.

        The block runs the newest token and all drafts but the last, so position t says what the model
        would have in the place of draft t.
        """
        logits = self.forward(torch.cat([self.last, drafts[:-1].long()]), commit_all=False)
        target, accepted = dn.dn_accept_greedy(logits.view(1, T, VOCAB), drafts.view(1, T))
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
    args = ap.parse_args()
    if args.prompt < 1:
        ap.error("a prompt has a token at least")
    model = HybridModel(cache=args.cache, max_tokens=args.prompt + T * (args.steps + 1))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    model.prompt(torch.randint(0, VOCAB, (args.prompt,), generator=g, device="cuda"))
    drafts = torch.randint(0, VOCAB, (T,), generator=g, device="cuda", dtype=torch.int32)
    for step in range(args.steps):
        target, accepted = model.verify(drafts)
        print("step %d: accepted %d of %d drafts, %d tokens cached; the model's own token is %d"
              % (step, int(accepted), T, int(model.kv_len), int(target[min(int(accepted), T - 1)])))
        # the next drafts: what the model itself had from the first rejected place on, then its last word again
        drafts = target[(torch.arange(T, device="cuda") + accepted).clamp(max=T - 1)].contiguous()


if __name__ == "__main__":
    main()
