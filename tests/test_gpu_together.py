"""The forks and the exact attention calls as one decoder would use them: samples of one prompt,
each step through a hybrid layer, an exact layer that keeps the prompt as a shared prefix, and
cross attention to one encoder output; then a beam step and a smaller batch."""
import pytest
import torch

import sparse_kv_caching_b200 as lola

pytestmark = pytest.mark.gpu
Hq, Hkv, d, Dh, ETA, LAM = 8, 2, 64, 32, 48, 40
PROMPT, STEPS, SOURCE, WIDTH = 640, 12, 333, Hq * d


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    lola.attention_check()


class Decoder:
    """Projections in torch; every attention through the library."""

    def __init__(self, room):
        g = torch.Generator("cuda").manual_seed(5)
        self.proj = [(torch.randn(WIDTH, (Hq + 2 * Hkv) * d, generator=g, device="cuda") / WIDTH**0.5).bfloat16() for _ in range(2)]
        self.wq = (torch.randn(WIDTH, WIDTH, generator=g, device="cuda") / WIDTH**0.5).bfloat16()
        W = (torch.randn(Hkv, d, Dh, generator=g, device="cuda") / d**0.5).bfloat16()
        self.layer = lola.LolaLayer(lola.make_config(room, Hq, Hkv, d, Dh, ETA, LAM, 64, "bf16", PROMPT), W)
        kv = torch.randn(1, SOURCE, 2, Hkv, d, generator=g, device="cuda").bfloat16()
        self.source = kv[:, :, 0], kv[:, :, 1]
        self.n = 0                                   # own tokens of the exact layer

    def qkv(self, x, i):
        z = (x @ self.proj[i]).view(*x.shape[:2], Hq + 2 * Hkv, d)
        return z[:, :, :Hq], z[:, :, Hq:Hq + Hkv], z[:, :, Hq + Hkv:]

    def finish(self, x):
        B = x.shape[0]
        k, v = (s.expand(B, -1, -1, -1) for s in self.source)
        y = lola.cross_attention((x @ self.wq).view(B, -1, Hq, d), k, v)
        x = x + y.reshape(x.shape)
        return x / x.float().square().mean(-1, keepdim=True).sqrt().to(x.dtype)

    def prompt(self, x, shared):
        """x [B, PROMPT, WIDTH]; shared: the exact layer keeps sequence 0's keys as the prefix of all."""
        q, k, v = (z.contiguous() for z in self.qkv(x, 0))
        x = x + self.layer.prefill(q, k, v).to(x.dtype).reshape(x.shape)
        q, k, v = self.qkv(x, 1)
        none = k[:, :0]
        y = lola.prefix_attention(q, none[0], none[0], k, v)
        if shared:
            self.prefix = k[0].contiguous(), v[0].contiguous()
            self.own = [torch.zeros(1, STEPS, Hkv, d, dtype=x.dtype, device="cuda") for _ in range(2)]
        else:
            self.prefix = none[0].contiguous(), none[0].contiguous()
            pad = torch.zeros(x.shape[0], STEPS, Hkv, d, dtype=x.dtype, device="cuda")
            self.own = [torch.cat([z, pad], 1) for z in (k, v)]
            self.n = PROMPT
        return self.finish(x + y.reshape(x.shape))

    def fork(self, parents):
        self.layer.fork(parents)
        self.own = [z[parents.long()].contiguous() for z in self.own]

    def step(self, x):
        q, k, v = (z[:, 0].contiguous() for z in self.qkv(x, 0))
        x = x + self.layer.decode(q, k, v).to(x.dtype).reshape(x.shape)
        q, k, v = self.qkv(x, 1)
        self.own[0][:, self.n], self.own[1][:, self.n] = k[:, 0], v[:, 0]
        self.n += 1
        y = lola.prefix_attention(q, *self.prefix, *self.own,
                                  own_len=torch.full((x.shape[0],), self.n, dtype=torch.int32, device="cuda"))
        return self.finish(x + y.reshape(x.shape))


def test_samples_beams_and_a_smaller_batch():
    """A forked batch with a shared prefix against a batch that prefilled and kept every copy: the
    same mathematics through other splits of the keys.  Tolerance: each attention output is rounded to
    bf16 (half a step, 2^-8) on both sides and every step feeds the next; 3 roundings a layer, two
    sides, and the normalisation keeps the scale, so 2^-8 x 6 x (steps) of the largest value."""
    g = torch.Generator("cuda").manual_seed(1)
    prompt = torch.randn(1, PROMPT, WIDTH, generator=g, device="cuda").bfloat16()
    N = 20
    a, b = Decoder(N), Decoder(N)
    a.layer.set_batch(1)
    xa = a.prompt(prompt, True)[:, -1:]
    xb = b.prompt(prompt.expand(N, -1, -1).contiguous(), False)[:, -1:]
    a.fork(torch.zeros(N, dtype=torch.int32, device="cuda"))
    xa = xa.expand(N, -1, -1)
    plans = {4: [i * 7 % 20 for i in range(20)], 8: [3, 3, 1, 17, 4, 9]}
    for t in range(STEPS):
        if t in plans:
            p = torch.tensor(plans[t], dtype=torch.int32, device="cuda")
            a.fork(p)
            b.fork(p)
            xa, xb = xa[p.long()], xb[p.long()]
        noise = torch.randn(xa.shape, generator=g, device="cuda").bfloat16()      # the samples differ
        xa, xb = a.step(xa + noise), b.step(xb + noise)
        off = float((xa.double() - xb.double()).abs().max() / xb.double().abs().max())
        assert off <= 2.0**-8 * 6 * (t + 1), (t, off)
    assert xa.shape[0] == 6 and torch.isfinite(xa.double()).all()
    a.layer.check()
