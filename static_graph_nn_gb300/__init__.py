"""GB300 training-step library: one full training step (forward, backward,
SGD/Adam update) of a typed static graph in hand-written sm_103a CUDA, behind
the C ABI of include/mg.h.  ``binding`` is the ctypes layer; ``workloads``
holds the seeded synthetic workloads."""
from .binding import (GradList, Plan, embedding_backward, embedding_forward,  # noqa: F401
                      embedding_workspace_bytes, grouped_linear_backward_input,
                      grouped_linear_backward_weight, grouped_linear_forward,
                      grouped_linear_status, grouped_linear_workspace_bytes, load)
