"""What a decode loop's requests hold, kept outside the cache, and their attention in double precision."""
import torch


class History:
    def __init__(self, batch):
        self.keys, self.values = [[] for _ in range(batch)], [[] for _ in range(batch)]

    def add(self, k, v, new):
        """new[b] rows of k and v [tokens, heads, D] to request b, request after request."""
        at = 0
        for b, n in enumerate(new):
            self.keys[b].append(k[at:at + n].double().cpu())
            self.values[b].append(v[at:at + n].double().cpu())
            at += n

    def attention(self, q):
        """(out, bound) [batch, q_heads, D] of q (16 bits; scale 1 / sqrt(D)).

        The bound is the output's rounding (2^-8 bf16, 2^-11 fp16), the scores' (fp32 sums of D products and
        a power of two: 4 ds of sum p|v|) and the sums' (2^-23 a token, weights within 2^-16).
        """
        u, q = 2.0 ** -8 if q.dtype is torch.bfloat16 else 2.0 ** -11, q.double().cpu()
        out, tol = torch.zeros_like(q), torch.zeros_like(q)
        d = q.shape[2]
        for b in range(q.shape[0]):
            k, v = torch.cat(self.keys[b]), torch.cat(self.values[b])
            if not len(k):
                continue
            for i in range(q.shape[1]):
                h = i * k.shape[1] // q.shape[1]
                s = k[:, h] @ q[b, i] * d ** -0.5
                p = torch.softmax(s, 0)
                out[b, i] = p @ v[:, h]
                ds = (d + 8) * 2.0 ** -23 * (k[:, h].abs() @ q[b, i].abs()).max() * d ** -0.5 + 2.0 ** -20 * (1 + s.abs().max())
                tol[b, i] = u * out[b, i].abs() + (4 * ds + 2.0 ** -16 + len(k) * 2.0 ** -23) * (p @ v[:, h].abs()) + 2.0 ** -25
        return out, tol
