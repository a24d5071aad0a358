"""Newton-Schulz orthogonalization for AMD Instinct MI355X (gfx950).

Python face of ``libnsortho.so``: the standard and Gram forms of quintic
Newton-Schulz (Muon's approximate polar factor), a batched launcher for
equal-shape expert matrices, the ROOT soft-threshold split, ROOT's per-shape
coefficient schedules (fitted on the host, run through the per-step
coefficient arrays) and a whole Muon step (momentum, orthogonalization,
weight update).  Beside it stand the operators that give the parameters Muon
leaves out their gradients: embedding, layer norm and the output projection's
softmax cross entropy, forward and backward.  The HIP
library does all the work; this package only marshals arguments.
"""

from .flops import gram_flops, ns_flops, standard_flops
from ._binding import (NS_MAX_STEPS, TUNED_ABC, NSError, lib, muon_step,
                       muon_workspace_size, orthogonalize,
                       orthogonalize_batched, orthogonalize_grouped,
                       orthogonalize_static, grouped_workspace_size,
                       plan_kernels,
                       soft_threshold_split, status_code, status_string,
                       workspace_size)
from ._training import (embedding, embedding_backward,
                        embedding_workspace_size, layer_norm,
                        layer_norm_backward, layer_norm_workspace_size,
                        linear_cross_entropy, linear_cross_entropy_backward,
                        linear_cross_entropy_workspace_size,
                        plan_linear_cross_entropy)
from .coeffs import fit_coefficients, root_coefficients

__all__ = [
    "NS_MAX_STEPS", "TUNED_ABC", "NSError", "lib", "muon_step",
    "muon_workspace_size", "orthogonalize",
    "orthogonalize_batched", "orthogonalize_grouped", "orthogonalize_static",
    "grouped_workspace_size", "plan_kernels", "soft_threshold_split",
    "status_code", "status_string",
    "workspace_size", "embedding", "embedding_backward",
    "embedding_workspace_size", "layer_norm", "layer_norm_backward",
    "layer_norm_workspace_size", "linear_cross_entropy",
    "linear_cross_entropy_backward", "linear_cross_entropy_workspace_size",
    "plan_linear_cross_entropy",
    "gram_flops", "ns_flops", "standard_flops",
    "fit_coefficients", "root_coefficients",
]
