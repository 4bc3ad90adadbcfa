"""fp64 logits processing: penalties for repeated tokens, biases, masks.

For token x of a row, in this order: with c the occurrences of x in the
generated part of the history and on the row's path,
  z = z / rho if z > 0 else z * rho    where c > 0 or x is in the prompt part
  z = z - frequency * c - presence * [c > 0]
  z = z + bias (of a token listed twice, the last entry)
  z = -inf where the mask forbids x.
"""
import numpy as np


def process_row(z, prompt, generated, path, rho, presence, frequency, bias=(), allowed=None):
    """The processed fp64 row, and the largest magnitude each value took on the way."""
    z = np.array(z, np.float64)
    V = z.shape[0]
    ok = lambda t: [x for x in t if 0 <= x < V]
    c = np.bincount(ok(list(generated) + list(path)), minlength=V).astype(np.float64)
    seen = (c > 0) | (np.bincount(ok(prompt), minlength=V) > 0)
    big = np.abs(z)
    z = np.where(seen, np.where(z > 0, z / rho, z * rho), z)
    big = np.maximum(big, np.abs(z))
    z = z - frequency * c
    big = np.maximum(big, np.maximum(np.abs(z), np.abs(frequency * c)))
    z = z - presence * (c > 0)
    big = np.maximum(big, np.abs(z))
    add = np.zeros(V)
    for x, y in bias:
        if 0 <= x < V:
            add[x] = y
    z = z + add
    big = np.maximum(big, np.abs(z))
    if allowed is not None:
        z[~allowed] = -np.inf
    return z, big
