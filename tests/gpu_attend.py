"""Attention in 64 bits on the GPU, from the definition, for the tests: one head at a time."""
import torch


def attend(q, k, v, see):
    """q [t, hq, d], k and v [n, hkv, d], see [t, n] (which keys each query sees).

    Returns, as float64 numpy arrays, o [t, hq, d], the sums of w |v| and the largest sum of |q k| / sqrt(d)
    of each row: what the tolerances are made of.  A row that sees nothing is 0."""
    t, hq, d = q.shape
    group = hq // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    o, absv = torch.zeros_like(q), torch.zeros_like(q)
    size = torch.zeros((t, hq, 1), dtype=torch.float64, device=q.device)
    some = see.any(1)
    if k.shape[0] and bool(some.any()):
        for h in range(hq):
            kk, vv = k[:, h // group], v[:, h // group]
            x = (q[:, h] @ kk.T / d ** 0.5).masked_fill(~see, float("-inf"))
            m = x.amax(1, keepdim=True)
            w = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
            w = torch.where(some[:, None], w / w.sum(1, keepdim=True), torch.zeros_like(w))
            o[:, h], absv[:, h] = w @ vv, w @ vv.abs()
            size[:, h, 0] = (q[:, h].abs() @ kk.abs().T / d ** 0.5).masked_fill(~see, 0.0).amax(1)
    return o.cpu().numpy(), absv.cpu().numpy(), size.cpu().numpy()


def seen(t, n, window, sinks, device="cuda"):
    """Which of n keys the queries at n - t .. n - 1 see."""
    p = torch.arange(n - t, n, device=device)[:, None]
    j = torch.arange(n, device=device)
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see
