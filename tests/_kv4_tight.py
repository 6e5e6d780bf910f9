"""Attention in 64 bits with a tolerance that follows the weights' own sum, so
that long prefixes are held to as many bits as short ones."""
import torch

from _kv4_util import up
from oracle import kv4 as okv4


def tight64(q, cache, T, seen, scale, k_global, v_global, dev):
    """(out, tolerance) of one request: q bf16 tensor [rows][Hq][128], cache the
    host bytes, seen bool [rows][rows].

    With p a slot's share of the row's weights, w its weight relative to the
    row's largest and l the sum of the w:
    * the output to bf16, half a step: 2^-8 |o|;
    * a weight to f16, once more where the row's maximum moves in the middle of
      a tile, and a partial O / l to f16: half a step 2^-11 each, so 3 * 2^-11
      of sum p |v|;
    * a weight below f16's normal range: half a step is 2^-25 there, twice, of a
      scale on which the running maximum has 2^7 or more: 2^-31 of w = 1, so
      n 2^-31 max |v| / l over n slots;
    * a partial O / l below it: 2^-25 in units of code * scale;
    * scores in fp32, 132 terms of at most 2^-23 each (products and partial
      sums; the tensor unit may truncate, a whole step) of sum |q| |k| * scale,
      in the weight and in the sum of weights; 2^-20 for the exponential and the
      rest of the fp32 arithmetic."""
    rows, Hq, _ = q.shape
    Hkv, n = cache[0].shape[0], T + rows
    G = Hq // Hkv
    k = up(okv4.values(cache[0][:, :n], cache[1][:, :n], k_global), dev)
    v = up(okv4.values(cache[2][:, :n], cache[3][:, :n], v_global), dev)
    vis = torch.cat((torch.ones(rows, T, dtype=torch.bool), torch.from_numpy(seen)), 1).to(dev)
    o, tol = torch.zeros((2, rows, Hq, 128), dtype=torch.float64, device=dev)
    for h in range(Hq):
        x, kh, vh = q[:, h].double(), k[h // G].double(), v[h // G].double()
        s = (x @ kh.t() * scale).masked_fill(~vis, -torch.inf)
        m = s.amax(-1, keepdim=True)
        w = torch.exp(s - torch.where(m > -torch.inf, m, torch.zeros_like(m)))
        l = w.sum(-1, keepdim=True)
        l = torch.where(l > 0, l, torch.ones_like(l))
        ds = (x.abs() @ kh.abs().t()).masked_fill(~vis, 0).amax(-1, keepdim=True) * scale * 132 * 2 ** -23
        o[:, h] = w @ vh / l
        spread, vmax = w @ vh.abs() / l, vh.abs().amax(0)
        tol[:, h] = (2 ** -8 * o[:, h].abs() + spread * (3 * 2 ** -11 + 2 * ds + 2 ** -20) + n * 2 ** -31 * vmax / l
                     + 2 ** -25 * v_global)
    return o, tol
