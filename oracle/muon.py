"""Float64 oracle of the orthogonalised step (include/salr.h, salr_muon_step),
from its definition: the Newton-Schulz steps on X itself."""

import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalise(u, eps=1e-7, steps=5, coefficients=COEFFICIENTS):
    """X after `steps` steps from u / (|u| + eps)."""
    a, b, c = coefficients
    X = u / (np.sqrt((u * u).sum()) + eps)
    if X.shape[0] > X.shape[1]:
        X = X.T
    for _ in range(steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X if X.shape == u.shape else X.T


def step(p, g, m, lr, momentum=0.95, nesterov=True, weight_decay=0.0, eps=1e-7, steps=5, coefficients=COEFFICIENTS,
         grad_scale=1.0, lr_scale=1.0):
    """(p, m, u) after one step."""
    g = g * grad_scale
    m = momentum * m + g
    u = g + momentum * m if nesterov else m
    return p * (1 - lr * weight_decay) - lr * lr_scale * orthogonalise(u, eps, steps, coefficients), m, u


def growth(s, steps=5, coefficients=COEFFICIENTS):
    """What a direction of the update whose squared singular value is s (of a
    unit-norm update) is multiplied with in all."""
    a, b, c = coefficients
    grow = np.ones_like(s)
    for _ in range(steps):
        now = s * grow * grow
        grow = grow * (a + b * now + c * now * now)
    return grow
