"""Serving with the 4-bit KV cache: prompts written and attended to in chunks,
several samples forked from each, single tokens decoded for all of them, pages
that fell out of the window given back and the pool packed on the way.

    python -m examples.kv_serving [--fmt nvfp4] [--steps 48] [--samples 3]

The model is a small random decoder (attention layers alone), so that what is
printed is about the cache: the pages in use over time, and how far the logits
are from those of the same tokens over keys and values kept in BF16.
"""
import argparse

import torch

import block_scaled_bit_fp4_amd as fp4

HEADS, KV_HEADS, DIM, WIDTH, VOCAB, LAYERS, PAGE = 8, 2, 64, 256, 512, 2, 32


class Model:
    """Attention layers with residuals; keys and values are views of one fused
    projection, as kv_append and kv_attention take them."""

    def __init__(self, seed, device):
        g = torch.Generator().manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g) / shape[-2] ** 0.5).to(device, torch.bfloat16)

        self.embed = w(VOCAB, WIDTH) * VOCAB ** 0.5
        self.qkv = [w(WIDTH, (HEADS + 2 * KV_HEADS) * DIM) for _ in range(LAYERS)]
        self.out = [w(HEADS * DIM, WIDTH) for _ in range(LAYERS)]

    def project(self, x, layer):
        y = (torch.nn.functional.rms_norm(x, (WIDTH,)) @ self.qkv[layer]).view(len(x), -1, DIM)
        return y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:]

    def run(self, tokens, attend):
        """Logits of the tokens; attend(layer, q, k, v) is the attention of a layer."""
        x = self.embed[tokens]
        for layer in range(LAYERS):
            x = x + attend(layer, *self.project(x, layer)).reshape(len(x), -1) @ self.out[layer]
        return torch.nn.functional.rms_norm(x, (WIDTH,)).float() @ self.embed.float().t()


class Pool:
    """A cache with its tables: rows of sequences, lengths, page counts."""

    def __init__(self, rows, pages, columns, fmt, device, window=0, sinks=0):
        # Hadamard-rotated rows; NVFP4 factors for values up to 12
        self.cache = fp4.new_kv_cache(pages, PAGE, KV_HEADS, DIM, fmt, LAYERS, k_scale=12 / 2688.0,
                                      v_scale=12 / 2688.0, rht=True, device=device)
        self.table = torch.full((rows, columns), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.window, self.sinks, self.device = window, sinks, device

    def grow(self, rows, n):
        """n more tokens for each of `rows`: the lowest free pages for those that begin one."""
        free = iter((self.refs == 0).nonzero().flatten().tolist())
        for r in rows:
            have = int(self.lens[r])
            for col in range(-(-have // PAGE), -(-(have + n) // PAGE)):
                page = next(free)
                self.table[r, col] = page
                self.refs[page] = 1
            self.lens[r] = have + n

    def step(self, model, rows, tokens):
        """`tokens` [rows, n]: the next tokens of these rows; their logits."""
        n = tokens.shape[1]
        self.grow(rows, n)
        at = torch.tensor(rows, device=self.device)
        batch = fp4.KVBatch(self.table[at], self.lens[at],
                            torch.arange(len(rows) + 1, dtype=torch.int32, device=self.device) * n, n)

        def attend(layer, q, k, v):
            fp4.kv_append(self.cache, k, v, batch, layer)
            return fp4.kv_attention(q, self.cache, batch, layer, window=self.window, sinks=self.sinks)

        return model.run(tokens.flatten(), attend).view(len(rows), n, VOCAB)

    def ids(self, rows):
        return torch.tensor(rows, dtype=torch.int32, device=self.device)

    def fork(self, parents, children):
        failed = fp4.kv_fork(self.cache, self.table, self.lens, self.refs, self.ids(parents), self.ids(children))
        if int(failed):
            raise RuntimeError("no free page for %d forks" % int(failed))

    def give_back(self, rows, window=0):
        fp4.kv_free(self.table, self.lens, self.refs, self.ids(rows), PAGE, window=window,
                    sinks=self.sinks if window else 0)

    def pack(self):
        return int(fp4.kv_compact(self.cache, self.table, self.refs)[1])


def serve(fmt="nvfp4", steps=48, samples=3, prompts=(200, 77, 130), chunk=64, window=128, sinks=4, pack_every=8,
          seed=0, device="cuda", say=lambda *a: None):
    """Returns the sampled tokens [sequences, steps], their logits, and the pages in use at each packing."""
    model = Model(seed, device)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    n, rows = len(prompts), len(prompts) * (1 + samples)
    pool = Pool(rows, rows * (-(-max(prompts) // PAGE) + 2) + 64, -(-(max(prompts) + steps) // PAGE), fmt, device,
                window, sinks)
    texts = [torch.randint(VOCAB, (m,), generator=g, device=device) for m in prompts]
    last = []
    for r, text in enumerate(texts):  # every prompt in chunks
        for part in text.split(chunk):
            logits = pool.step(model, [r], part[None])
        last.append(logits[:, -1])
    children = list(range(n, rows))
    parents = [(c - n) // samples for c in children]
    pool.fork(parents, children)
    pool.give_back(range(n))  # the samples hold the prompts' pages now
    logits = torch.cat(last)[parents]
    tokens, seen, used = [], [], []
    for i in range(steps):
        seen.append(logits)
        tokens.append(torch.multinomial(torch.softmax(logits, -1), 1, generator=g))
        logits = pool.step(model, children, tokens[-1])[:, -1]
        if window:
            pool.give_back(children, window)
        if pack_every and (i + 1) % pack_every == 0:
            used.append(pool.pack())
            say("%3d tokens a sample: %d of %d pages in use" % (i + 1, used[-1], len(pool.refs)))
    return model, texts, parents, torch.cat(tokens, 1), torch.stack(seen, 1), used


def plain_logits(model, tokens, window, sinks):
    """Logits of one sequence with keys and values as they are, in 32 bits."""
    t = torch.arange(len(tokens), device=tokens.device)
    see = t[None] <= t[:, None]
    if window:
        see &= (t[None] > t[:, None] - window) | (t[None] < sinks)

    def attend(layer, q, k, v):
        k, v = (x.float().repeat_interleave(HEADS // KV_HEADS, 1).transpose(0, 1) for x in (k, v))
        s = (q.float().transpose(0, 1) @ k.transpose(1, 2).contiguous()) / DIM ** 0.5
        p = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
        return (p @ v).transpose(0, 1).to(torch.bfloat16)

    return model.run(tokens, attend)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--fmt", default="nvfp4", choices=("nvfp4", "mxfp4", "mxfp4_oas"))
    ap.add_argument("--steps", type=int, default=48)
    ap.add_argument("--samples", type=int, default=3)
    a = ap.parse_args()
    window, sinks = 128, 4
    model, texts, parents, tokens, logits, _ = serve(a.fmt, a.steps, a.samples, window=window, sinks=sinks, say=print)
    errs = []
    for c, p in enumerate(parents):
        want = plain_logits(model, torch.cat((texts[p], tokens[c])), window, sinks)[len(texts[p]) - 1:-1]
        errs.append(float((logits[c] - want).norm() / want.norm()))
    print("logits against keys and values in BF16: relative error %.4f (largest of %d samples)" % (max(errs), len(errs)))


if __name__ == "__main__":
    main()
